"""The attention, norm and rotation entry points on the CPU: arguments that
they reject before any device work, and the mirrors of their structs."""
import ctypes
import os

import pytest

import submanifold_sparse_convolution_device_amd as sp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every case fails validation first


def _status(fn, *a):
    with pytest.raises(sp.SpconvError) as e:
        fn(*a)
    return e.value.name


def _attention(**changes):
    a = sp.spconv_attention(q=FAKE, k=2 * FAKE, v=3 * FAKE, q_row_stride=128, q_head_stride=32, k_row_stride=64, k_head_stride=32,
                            v_row_stride=64, v_head_stride=32, cu_q=FAKE, cu_k=FAKE, total_q=10, total_k=12, batch=1, heads=4,
                            kv_heads=2, head_dim=32, left=-1, right=-1, scale=0.2, dtype=2)
    for k, v in changes.items():
        setattr(a, k, v)
    return a


def _forward(**changes):
    out, lse = changes.pop("out", 4 * FAKE), changes.pop("lse", 5 * FAKE)
    return _status(sp.spconv_attention_forward, _attention(**changes), out, lse, 0)


def test_attention_rejects():
    bad = "SPCONV_ERR_INVALID_ARG"
    for c in ({"q": 0}, {"k": 0}, {"v": 0}, {"cu_q": 0}, {"cu_k": 0}, {"out": 0}, {"lse": 0}, {"q": FAKE + 8}, {"out": 4 * FAKE + 2},
              {"lse": 5 * FAKE + 2}, {"cu_k": FAKE + 1}, {"heads": 5}, {"heads": 0}, {"kv_heads": 0}, {"kv_heads": -2}, {"batch": -1},
              {"total_q": -1}, {"total_k": -1}, {"total_q": 1 << 40}, {"total_k": (1 << 30) + 1}, {"total_q": 1 << 30}, {"scale": 0.0},
              {"scale": float("nan")}, {"q_row_stride": 12}, {"k_row_stride": -64}, {"v_head_stride": 1}, {"k_row_stride": 1 << 40},
              {"out": FAKE}, {"out": 2 * FAKE + 64}, {"lse": 3 * FAKE}, {"lse": 4 * FAKE + 16}):
        assert _forward(**c) == bad, c
    for c in ({"dtype": 3}, {"dtype": -1}, {"head_dim": 0}, {"head_dim": 12}, {"head_dim": 136}):
        assert _forward(**c) == "SPCONV_ERR_UNSUPPORTED", c
    assert sp.STATUS[sp.lib().spconv_attention_forward(None, FAKE, FAKE, None)] == bad


def test_attention_backward_rejects():
    def grads(**changes):
        g = sp.spconv_attention_gradients(grad_out=6 * FAKE, grad_out_row_stride=128, grad_out_head_stride=32, grad_q=7 * FAKE,
                                          grad_q_row_stride=128, grad_q_head_stride=32, grad_k=8 * FAKE, grad_k_row_stride=64,
                                          grad_k_head_stride=32, grad_v=9 * FAKE, grad_v_row_stride=64, grad_v_head_stride=32)
        for k, v in changes.items():
            setattr(g, k, v)
        return g

    f = sp.spconv_attention_backward
    for c in ({"grad_out": 0}, {"grad_q": 0}, {"grad_k": 0}, {"grad_v": 0}, {"grad_q": FAKE}, {"grad_k": 2 * FAKE}, {"grad_v": 4 * FAKE},
              {"grad_v": 5 * FAKE}, {"grad_q": 6 * FAKE}, {"grad_k": 7 * FAKE}, {"grad_v": 8 * FAKE}, {"grad_q": 7 * FAKE + 4},
              {"grad_q_row_stride": 0}, {"grad_k_head_stride": 0}, {"grad_k_head_stride": 16}, {"grad_v_row_stride": 40}):
        assert _status(f, _attention(), 4 * FAKE, 5 * FAKE, grads(**c), 0) == "SPCONV_ERR_INVALID_ARG", c
    a = _attention()
    assert sp.STATUS[sp.lib().spconv_attention_backward(ctypes.byref(a), 4 * FAKE, 5 * FAKE, None, None)] == "SPCONV_ERR_INVALID_ARG"
    assert _status(f, _attention(head_dim=4), 4 * FAKE, 5 * FAKE, grads(), 0) == "SPCONV_ERR_UNSUPPORTED"


def _norm(**changes):
    a = sp.spconv_norm_rotary(q=FAKE, k=2 * FAKE, q_row_stride=128, q_head_stride=32, k_row_stride=64, k_head_stride=32,
                              q_weight=3 * FAKE, k_weight=3 * FAKE, table=4 * FAKE, positions=5 * FAKE, position_row_stride=3, rows=10,
                              q_heads=4, k_heads=2, head_dim=32, rotary_dim=24, axes=3, extent=100, interleaved=0, eps=1e-6, dtype=2)
    for k, v in changes.items():
        setattr(a, k, v)
    return a


def test_norm_rotary_rejects():
    def forward(q_out=6 * FAKE, k_out=7 * FAKE, strides=(128, 32, 64, 32), **changes):
        return _status(sp.spconv_norm_rotary_forward, _norm(**changes), q_out, strides[0], strides[1], k_out, strides[2], strides[3], 0)

    for c in ({"q": 0}, {"k": 0}, {"q_out": 0}, {"k_out": 0}, {"table": 0}, {"positions": 0}, {"q": FAKE + 2}, {"q_weight": 3 * FAKE + 2},
              {"table": 4 * FAKE + 4}, {"positions": 5 * FAKE + 2}, {"rows": -1}, {"rows": 1 << 31}, {"q_heads": -1}, {"k_heads": -1},
              {"rotary_dim": 34}, {"rotary_dim": -2}, {"axes": 0}, {"axes": 5}, {"extent": 0}, {"extent": 1 << 25}, {"interleaved": 2},
              {"eps": -1.0}, {"eps": float("inf")}, {"position_row_stride": -1}, {"q_row_stride": 4}, {"q_out": 2 * FAKE},
              {"k_out": 6 * FAKE}, {"q_out": FAKE, "strides": (192, 32, 64, 32)}, {"strides": (64, 32, 64, 32)}, {"strides": (128, 0, 64, 32)}):
        assert forward(**c) == "SPCONV_ERR_INVALID_ARG", c
    for c in ({"dtype": 5}, {"head_dim": 20}, {"head_dim": 160}, {"rotary_dim": 20}):
        assert forward(**c) == "SPCONV_ERR_UNSUPPORTED", c
    assert sp.STATUS[sp.lib().spconv_norm_rotary_forward(None, FAKE, 1, 1, FAKE, 1, 1, None)] == "SPCONV_ERR_INVALID_ARG"

    def backward(**changes):
        g = sp.spconv_norm_rotary_gradients(grad_q_out=6 * FAKE, grad_k_out=7 * FAKE, grad_q_out_row_stride=128, grad_q_out_head_stride=32,
                                            grad_k_out_row_stride=64, grad_k_out_head_stride=32, grad_q=8 * FAKE, grad_k=9 * FAKE,
                                            grad_q_row_stride=128, grad_q_head_stride=32, grad_k_row_stride=64, grad_k_head_stride=32,
                                            grad_q_weight=10 * FAKE, grad_k_weight=11 * FAKE)
        for k, v in changes.items():
            setattr(g, k, v)
        return _status(sp.spconv_norm_rotary_backward, _norm(), g, 0)

    for c in ({"grad_q_out": 0}, {"grad_k_out": 0}, {"grad_q": 0}, {"grad_k": 0}, {"grad_q": FAKE}, {"grad_k": 8 * FAKE}, {"grad_q": 7 * FAKE},
              {"grad_q_weight": 10 * FAKE + 1}, {"grad_q_row_stride": 0}, {"grad_k_head_stride": 8}):
        assert backward(**c) == "SPCONV_ERR_INVALID_ARG", c


def test_rotary_table_rejects():
    f = sp.spconv_rotary_table
    for a in ((0, 4, 4, 1e4, 1.0), (FAKE + 4, 4, 4, 1e4, 1.0), (FAKE, 0, 4, 1e4, 1.0), (FAKE, 4, 0, 1e4, 1.0), (FAKE, 4, 4, 0.0, 1.0),
              (FAKE, 4, 4, float("inf"), 1.0), (FAKE, 4, 4, 1e4, float("nan")), (FAKE, 1 << 25, 4, 1e4, 1.0)):
        assert _status(f, *a, 0) == "SPCONV_ERR_INVALID_ARG", a


def test_struct_mirrors_have_the_c_sizes():
    """The ctypes mirrors against the compiler's sizes and offsets."""
    import subprocess
    import tempfile
    names = ("spconv_attention", "spconv_attention_gradients", "spconv_norm_rotary", "spconv_norm_rotary_gradients")
    lines = []
    for n in names:
        lines.append(f'printf("%zu", sizeof({n}));')
        lines += [f'printf(" %zu", offsetof({n}, {f}));' for f, _ in getattr(sp, n)._fields_]
        lines.append('printf("\\n");')
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"spconv.h\"\nint main(void) {" + "".join(lines) + "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "t.c"), "w") as f:
            f.write(src)
        exe = os.path.join(d, "t")
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, os.path.join(d, "t.c")], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    for n, line in zip(names, got):
        cls = getattr(sp, n)
        assert [int(v) for v in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_], n


def test_packed_arguments_have_the_structs_layout():
    """The packed bytes of the torch front end against the struct mirrors."""
    for pack, cls in ((sp._PACK_ATTENTION, sp.spconv_attention), (sp._PACK_ATTENTION_GRADIENTS, sp.spconv_attention_gradients),
                      (sp._PACK_NORM_ROTARY, sp.spconv_norm_rotary),
                      (sp._PACK_NORM_ROTARY_GRADIENTS, sp.spconv_norm_rotary_gradients)):
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(pack.pack(*values))
        assert pack.size == ctypes.sizeof(cls)
        assert [getattr(got, f) for f, _ in cls._fields_] == values


def test_entry_points_under_sanitizers():
    """This file's tests against the library's host code built with
    AddressSanitizer and UndefinedBehaviorSanitizer."""
    import subprocess
    import sys
    if os.environ.get("SPCONV_LIB_PATH"):
        pytest.skip("already in the sanitized run")
    sanitized_build = pytest.importorskip("sanitized_build")
    runtime = sanitized_build.clang_asan_runtime()
    if not runtime or not os.path.exists(sanitized_build.HIPCC):
        pytest.skip("no hipcc or clang ASan runtime")
    env = dict(os.environ, LD_PRELOAD=runtime, SPCONV_LIB_PATH=sanitized_build.build_library(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.basename(__file__), "-q", "-x", "-s", "-p", "no:cacheprovider",
                        "--deselect", "test_attention_abi_host.py::test_struct_mirrors_have_the_c_sizes"],
                       cwd=os.path.dirname(os.path.abspath(__file__)), env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "runtime error" not in out and "ERROR: AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
