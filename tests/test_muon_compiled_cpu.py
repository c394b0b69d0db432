"""What the compiler made of the Newton-Schulz products. Their matrix
instructions are inline assembly, whose latency the compiler does not know:
none of its own instructions may touch an accumulator between a product and
the wait behind the loop."""

import os
import re
import subprocess

import pytest

from zero_sharded_mixed_tensor_amd import build

INSTR = re.compile(r"^\s+([a-z][a-z0-9_]+)(\s.*)?$")


def early_accesses(lines):
    """Instructions (one function's, in the order they lie) that read or write
    an accumulator behind a matrix instruction and before the wait; but for
    the zeros it starts from, whose block may lie anywhere."""
    bad, pending = [], False
    for line in lines:
        m = INSTR.match(line.split(";")[0])
        if not m:
            continue
        op, args = m.group(1), m.group(2) or ""
        acc = re.search(r"\ba(\d|\[)", args)
        if op.startswith("v_mfma"):
            pending = True
        elif op == "s_nop" and args.strip() == "15":
            pending = False
        elif pending and acc and not re.match(r"v_accvgpr_write_b32 a\d+, 0$", (op + args).strip()):
            bad.append(line.strip())
    return bad


def test_the_check_sees_an_early_access():
    loop = ["\tv_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", "\ts_cbranch_scc0 .LBB0_1"]
    read = ["\tv_accvgpr_read_b32 v0, a0", "\tglobal_store_dwordx4 v[0:1], a[0:3], off"]
    assert early_accesses(loop + ["\ts_nop 15"] + read) == []
    assert len(early_accesses(loop + read + ["\ts_nop 15"])) == 2


def test_products_wait_before_their_accumulators_are_read(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "ns.s"
    cmd = [build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S",
           os.path.join(build.CSRC, "zds_newton_schulz.hip"), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    text = out.read_text()
    found = re.findall(r"^(_ZN3zds17ns_product_kernel\w+):\s.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S)
    assert len(found) >= 30
    for name, body in found:
        assert body.count("v_mfma") > 0 and "s_nop 15" in body, name
        assert early_accesses(body.splitlines()) == [], name
    # and they keep everything in registers
    sizes = re.findall(r"\.name:\s+(_ZN3zds17ns_product_kernel\w+).*?\.private_segment_fixed_size:\s+(\d+)", text, re.S)
    assert len(sizes) == len(found) and all(int(n) == 0 for _, n in sizes), sizes


def test_the_high_half_of_a_pair_is_rounded_one_way(tmp_path):
    """A number's high half is stored and taken off to form the low one: two
    uses that must see one rounding. An instruction that rounds an exact
    product straight to fp16 next to conversions of its fp32 value makes them
    two."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "ns.s"
    cmd = [build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S",
           os.path.join(build.CSRC, "zds_newton_schulz.hip"), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    kernels = re.findall(r"^(_ZN3zds\d+ns_\w+):\s.*?\n(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S)
    assert len(kernels) >= 50
    assert [name for name, body in kernels if "v_fma_mix" in body] == []
