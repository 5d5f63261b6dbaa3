"""An SM holds six CTAs of the kernels that take plain 16-bit activations over odd rows and keep their
inputs: as the compiler reports their registers (42, five CTAs, cost 3 % of the time)."""
import os
import re
import subprocess


def test_odd_rows_keep_six_ctas_an_sm(tmp_path):
    from loss_scaling_master_gb300 import build as B
    r = subprocess.run([B.nvcc(), *B.FLAGS, "-Xptxas", "-v", "-c", os.path.join(B.CSRC, "act_mx8.cu"), "-o",
                        str(tmp_path / "act.o")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    # act_fwd_elem<f16 or bf16, an activation, plain, kept, by eight blocks>
    found = re.findall(r"Compiling entry function '\S*act_fwd_elemILi[12]ELi[012]ELb0ELb1ELi8E.*?"
                       r"(\d+) bytes spill stores.*?Used (\d+) registers", r.stderr + r.stdout, re.S)
    assert len(found) == 6
    for spills, regs in found:
        # 256 threads a CTA, registers given out by 8 a thread
        assert spills == "0" and 6 * 256 * (-(-int(regs) // 8) * 8) <= 65536, found
