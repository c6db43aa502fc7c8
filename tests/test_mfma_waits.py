"""The waits between matrix products and the instructions that read their
sums, in the generated code of the attention kernels (CPU only: compiles them
to assembly).

The hardware does not hold a vector or memory instruction back that reads an
accumulator before its product is done; the compiler places the waits, and has
been seen to leave one out across blocks.  This walks every path from every
product to every reader of its registers and counts the wait states between.
"""
import concurrent.futures
import os
import re
import subprocess

import pytest

import submanifold_sparse_convolution_device_amd.build as lib_build

# States between an 8-pass product (32x32x16) and a reader.
NEED = 12


def _registers(operand):
    m = re.match(r"^-?\|?([av])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"^-?\|?([av])(\d+)\|?$", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


def early_reads(body):
    """(product, reader, states) of every read that may come too early."""
    code, labels = [], {}
    for line in body.split("\n"):
        line = line.split(";")[0].rstrip()
        if re.match(r"^\.LBB\S+:", line):
            labels[line.split(":")[0]] = len(code)
        elif line.startswith("\t") and line.strip() and not line.strip().startswith("."):
            parts = line.split(None, 1)
            code.append((parts[0], [x.strip() for x in parts[1].split(",")] if len(parts) > 1 else []))
    found = []
    for i, (op, operands) in enumerate(code):
        if "mfma" not in op:
            continue
        sums = _registers(operands[0])
        best, stack = {}, [(i + 1, 0)]
        while stack:
            j, states = stack.pop()
            if j >= len(code) or states >= NEED or best.get(j, NEED) <= states:
                continue
            best[j] = states
            o, a = code[j]
            if "mfma" in o:
                if _registers(a[0]) & sums:
                    continue  # summed on, or written anew: that product's own readers count
            elif o.startswith(("v_", "ds_", "buffer_", "global_", "scratch_")):
                # every operand, for these may write what they read; the first of a vector instruction is its result
                read = a if not o.startswith("v_") or "swap" in o else a[1:]
                if set().union(*map(_registers, read), set()) & sums:
                    found.append((op, o, states))
                    continue
            if o == "s_endpgm":
                continue
            if o == "s_branch":
                stack.append((labels[a[0]], states + 1))
                continue
            if o.startswith("s_cbranch"):
                stack.append((labels[a[0]], states + 1))
            stack.append((j + 1, states + (int(a[0], 0) + 1 if o == "s_nop" else 1)))
    return found


def _assembly(source, out):
    cmd = [lib_build.HIPCC, *lib_build.FLAGS, *lib_build.EXTRA_FLAGS.get(source, []), "-S", "--cuda-device-only",
           os.path.join(lib_build.CSRC, source), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        return f.read()


def test_the_walk_sees_a_missing_wait():
    product = "\tv_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], v[0:15]\n"
    read = "\tv_add_f32 v40, v15, v41\n"
    assert early_reads(product + "\ts_nop 7\n" + read)
    assert not early_reads(product + "\ts_nop 15\n" + read)
    # a short way and a long way to the same read
    two = (product + "\ts_cbranch_vccnz .LBB0_1\n\ts_nop 12\n.LBB0_1:\n" + read)
    assert [s for _, _, s in early_reads(two)] == [1]
    assert not early_reads(product + "\ts_nop 15\n\ts_cbranch_vccnz .LBB0_1\n\ts_nop 12\n.LBB0_1:\n" + read)


def test_attention_kernels_wait_for_their_products(tmp_path):
    if not os.path.exists(lib_build.HIPCC):
        pytest.skip("no hipcc")
    sources = ["attention.hip", "attention_backward.hip"]
    with concurrent.futures.ThreadPoolExecutor(len(sources)) as ex:
        texts = list(ex.map(lambda s: _assembly(s, str(tmp_path / (s + ".txt"))), sources))
    kernels = 0
    for text in texts:
        for m in re.finditer(r"^(_Z\S*):[^\n]*\n(.*?)\.end_amdhsa_kernel", text, re.S | re.M):
            kernels += "mfma" in m.group(2)
            assert not early_reads(m.group(2)), m.group(1)
    # 3 types x 8 head sizes x 3 workgroup sizes, forward and the two gradients
    assert kernels == 3 * 8 * 3 * 3
