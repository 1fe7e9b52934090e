"""The 8-bit norm's plan counts the CTAs that an SM holds by its kernels' registers: the numbers in
the source against the compiler's.  (A CTA too many is a second wave: with 96 registers counted
where a form takes 106, 65536 x 2048 with a full gate took 270 us where it takes 188.)"""
import os
import re
import subprocess

from top_routing_expert_moe_gb300 import build

SRC = os.path.join(build.CSRC, "norm_rows.cuh")
FORM = re.compile(r"block_norm_ring_kernelI13__nv_bfloat16Lb1EL\w*?(\d)ELi(\d+)ELb1E")


def test_registers_are_the_compilers(tmp_path):
    text = open(SRC).read()
    m = re.search(r"form_of\(a, false\) == FORM_ANY \? (\d+) : heavy \? (\d+) : (\d+)\)", text)
    assert m, "the plan's registers"
    names = re.search(r"enum Form \{(.*?)\};", text, re.S).group(1)
    forms = re.findall(r"\bFORM_\w+", re.sub(r"//[^\n]*", "", names))
    counted = dict.fromkeys(forms, int(m.group(3)))
    counted.update(FORM_ANY=int(m.group(1)), FORM_BOTH=int(m.group(2)))
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-Xptxas", "-v", "-c", os.path.join(build.CSRC, "norm_mx8.cu"),
                        "-o", str(tmp_path / "n.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    seen = set()
    for name, used in re.findall(r"Compiling entry function '(\S+)'.*?Used (\d+) registers", r.stderr, re.S):
        k = FORM.search(name)
        if not k or int(k.group(2)) > 512:           # (wider rows have an SM to themselves)
            continue
        form = forms[int(k.group(1))]
        seen.add(form)
        allocated = (int(used) + 7) // 8 * 8
        assert allocated <= counted[form], (form, k.group(2), used)
    assert seen >= {"FORM_ANY", "FORM_BOTH", "FORM_ADD", "FORM_ENTER"}
