"""Host side of the rotary positions and the 4-bit cache, without a GPU: the
axis helper, the refusals of every entry point, the struct's C layout, and
the test definitions' own round trip."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import _kvq
import workloads as wl
import paged_kv_gqa_attention_gb300 as qa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


def test_rope_axes():
    np.testing.assert_array_equal(qa.qa_rope_axes([64]), np.zeros(64))
    np.testing.assert_array_equal(qa.qa_rope_axes([16, 24, 24]), [0] * 16 + [1] * 24 + [2] * 24)
    np.testing.assert_array_equal(qa.qa_rope_axes([16, 16], head_dim=64), [0] * 16 + [1] * 16)
    inter = qa.qa_rope_axes([24, 20, 20], interleaved=True)
    np.testing.assert_array_equal(inter, [i % 3 if i < 60 else 0 for i in range(64)])
    assert [int((inter == a).sum()) for a in range(3)] == [24, 20, 20]
    np.testing.assert_array_equal(qa.qa_rope_axes([0, 64, 0, 0]), np.ones(64))


@pytest.mark.parametrize("sections, kw", [
    ([32, 31], {}), ([64, 1], {}), ([70, -6], {}), ([], {}), ([16] * 5, {}), ([40], dict(head_dim=80)),
    ([20, 22, 22], dict(interleaved=True)), ([0, 64], dict(interleaved=True)),
])
def test_rope_axes_refuses(sections, kw):
    with pytest.raises(qa.QAError):
        qa.qa_rope_axes(sections, **kw)


def test_rope_struct_has_the_c_layout(tmp_path):
    c = tmp_path / "layout.c"
    names = [n for n, _ in qa.qa_rope._fields_]
    c.write_text('#include "qa.h"\n#include <stdio.h>\nint main(void) { printf("%u", (unsigned)sizeof(qa_rope));\n'
                 + "".join(f'printf(" %u", (unsigned)offsetof(qa_rope, {n}));\n' for n in names) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(c), "-o",
                    str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(qa.qa_rope)] + [getattr(qa.qa_rope, n).offset for n in names]


def test_angles_are_reduced_to_half_a_turn(tmp_path):
    """Every position at the largest frequency, a radian a position, and at a few smaller ones: the fraction of a turn is
    in [-1/2, 1/2], where the hardware sine and cosine have their bound, and within 2^-24 of the true one (2^-25 for the
    rounding of a sum below 1, the other terms are below 2^-30)."""
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text('#include "rotary.cuh"\n#include <stdio.h>\n#include <stdlib.h>\nint main(int, char **v) {\n'
                   "    const double t = atof(v[1]);\n    const float hi = (float)t, lo = (float)(t - (double)hi);\n"
                   "    for (int p = 0; p < 1 << 18; ++p) {\n        const float f = qa::turn_fraction(p, hi, lo);\n"
                   "        fwrite(&f, sizeof f, 1, stdout);\n    }\n    return 0;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-I", os.path.join(ROOT, "paged_kv_gqa_attention_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    pos = np.arange(1 << 18, dtype=np.float64)
    for radians in (1.0, 1e4 ** (-2 / 128), 1e6 ** (-1 / 2), 0.5):
        t = radians / (2 * np.pi)
        got = np.frombuffer(subprocess.run([str(exe), repr(t)], stdout=subprocess.PIPE, check=True).stdout, np.float32)
        off = got - pos * t  # pos t to 2^-37: a whole number of turns from the fraction
        assert np.abs(off - np.rint(off)).max() <= 2.0 ** -24
        assert np.abs(got).max() <= 0.5


def params(**kw):
    p = qa.qa_attn_default_params()
    p.num_pages, p.max_pages_per_seq = 4, 4
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def rope(**kw):
    r = qa.qa_rope()
    r.theta, r.rms_eps, r.n_axes = 1e6, 1e-6, 1
    r.q_gain = r.k_gain = r.positions = 0x1000
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.byref(r)


def refused(status, word):
    assert status == -1, qa.qa_last_error()
    assert word in qa.qa_last_error(), qa.qa_last_error()


def test_rope_rows_refuses():
    def call(q=FAKE, ldq=0, k=FAKE, ldk=0, rows=3, qo=FAKE, ldqo=0, ko=FAKE, ldko=0, r=None, p=None):
        return qa._lib.qa_rope_rows(q, ldq, k, ldk, rows, qo, ldqo, ko, ldko, r or rope(), p or params())

    refused(call(q=None), "NULL")
    refused(call(ko=None), "NULL")
    refused(call(rows=-1), "rows")
    refused(call(q=ODD), "aligned")
    refused(call(p=params(head_dim=80)), "head_dim")
    refused(call(p=params(n_q_heads=0)), "head counts")
    refused(call(p=params(stable_metadata=3)), "stable_metadata")
    refused(call(p=params(abi_version=99)), "abi_version")
    refused(call(ldq=2047), "ldq")
    refused(call(ldk=1020), "ldk")
    refused(call(ldqo=4096), "row stride")
    refused(call(r=rope(theta=0.0)), "theta")
    refused(call(r=rope(theta=float("nan"))), "theta")
    refused(call(r=rope(rms_eps=0.0)), "rms_eps")
    refused(call(r=rope(q_gain=None)), "gain")
    refused(call(r=rope(q_gain=0x1004)), "aligned")
    refused(call(r=rope(n_axes=0)), "n_axes")
    refused(call(r=rope(n_axes=5)), "n_axes")
    refused(call(r=rope(positions=None)), "positions")
    axes = np.zeros(64, np.uint8)
    axes[63] = 1
    refused(call(r=rope(pair_axis=axes.ctypes.data)), "pair_axis[63]")
    assert qa._lib.qa_rope_rows(FAKE, 0, FAKE, 0, 3, FAKE, 0, FAKE, 0, None, params()) == -1
    assert call(rows=0) == 0  # nothing to do, nothing launched


def test_frequency_bases_below_one_are_refused():
    """Pairs would turn by more than a radian a position, past what the reduction of angles is exact for."""
    for theta in (0.99, 1e-30, -1.0, float("inf")):
        refused(qa._lib.qa_rope_rows(FAKE, 0, FAKE, 0, 3, FAKE, 0, FAKE, 0, rope(theta=theta), params()), "theta")
        refused(qa._lib.qa_kvq_decode_step(FAKE, 0, FAKE, FAKE, 0, rope(theta=theta), FAKE, FAKE, FAKE, FAKE, 1, FAKE, params()),
                "theta")


def test_more_pages_than_the_decode_numbers():
    for batch, wide in ((9, 2**27 - 1), (4096, 2**18 + 1)):
        p = params(max_pages_per_seq=wide)
        refused(qa._lib.qa_kvq_decode_attn(FAKE, FAKE, FAKE, FAKE, FAKE, batch, FAKE, p), "max_pages_per_seq")
        refused(qa._lib.qa_kvq_decode_step(FAKE, 0, FAKE, FAKE, 0, rope(), FAKE, FAKE, FAKE, FAKE, batch, FAKE, p),
                "max_pages_per_seq")
    p = params(max_pages_per_seq=2**18)
    assert qa._lib.qa_kvq_decode_attn(FAKE, FAKE, FAKE, FAKE, FAKE, 4096, FAKE, p) in (-1, -3)
    assert "max_pages_per_seq" not in qa.qa_last_error()  # no workspace, or no device


def test_pages_refuse():
    def write(k=FAKE, ldk=0, v=FAKE, ldv=0, cu=FAKE, past=FAKE, batch=2, total=5, table=FAKE, kp=FAKE, vp=FAKE, p=None):
        return qa._lib.qa_kvq_write(k, ldk, v, ldv, cu, past, batch, total, table, kp, vp, p or params())

    def read(kp=FAKE, vp=FAKE, table=FAKE, cu=FAKE, past=None, batch=2, total=5, k=FAKE, v=FAKE, p=None):
        return qa._lib.qa_kvq_read(kp, vp, table, cu, past, batch, total, k, v, p or params())

    for fn in (write, read):
        refused(fn(k=None), "NULL")
        refused(fn(cu=None), "NULL")
        refused(fn(batch=0), "batch")
        refused(fn(batch=4097), "batch")
        refused(fn(total=-1), "total_tokens")
        refused(fn(vp=ODD), "aligned")
        refused(fn(past=ctypes.c_void_p(0x1002)), "aligned")
        for field, bad in (("head_dim", 64), ("n_kv_heads", 9), ("n_q_heads", 24), ("page_size", 32), ("num_pages", 0),
                           ("max_pages_per_seq", 0)):
            refused(fn(p=params(**{field: bad})), "")
    refused(write(ldk=1016), "ldk")
    refused(write(ldv=1028), "ldv")


def test_decode_refuses():
    def attn(q=FAKE, batch=1, kp=FAKE, out=FAKE, p=None):
        return qa._lib.qa_kvq_decode_attn(q, kp, FAKE, FAKE, FAKE, batch, out, p or params())

    def step(q=FAKE, ldq=0, k=FAKE, ldkv=0, r=None, kp=FAKE, batch=1, out=FAKE, p=None):
        return qa._lib.qa_kvq_decode_step(q, ldq, k, FAKE, ldkv, r or rope(), kp, FAKE, FAKE, FAKE, batch, out, p or params())

    for fn in (attn, step):
        refused(fn(q=None), "NULL")
        refused(fn(kp=ODD), "aligned")
        refused(fn(batch=0), "batch")
        refused(fn(p=params(n_q_heads=32)), "n_q_heads")
        refused(fn(p=params(scale=-1.0)), "scale")
        assert fn() in (-1, -3)  # no workspace; without a GPU, no device
        assert "workspace" in qa.qa_last_error() or "device" in qa.qa_last_error()
    refused(step(k=None), "NULL")
    refused(step(k=ODD), "aligned")
    refused(step(ldq=1024), "ldq")
    refused(step(ldkv=12), "ldkv")
    refused(step(r=rope(q_gain=None, k_gain=None)), "gain")
    refused(step(r=rope(positions=None, n_axes=2)), "positions")
    refused(step(r=rope(positions=None), p=params(max_pages_per_seq=20000)), "positions")


def test_sizes():
    assert [qa.qa_kvq_page_bytes(h) for h in (1, 8)] == [1280, 10240]
    with pytest.raises(qa.QAError):
        qa.qa_kvq_page_bytes(9)
    with pytest.raises(qa.QAError):
        qa.qa_kvq_decode_workspace_size(0, 0)
    with pytest.raises(qa.QAError):
        qa.qa_kvq_decode_workspace_size(1, 17)  # past max_pages_per_seq * 16


def test_python_checks():
    torch = pytest.importorskip("torch")
    rows = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(3, 10240, dtype=torch.uint8)
    cu, table = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages must be a CUDA tensor"):
        qa.qa_kvq_write(rows, rows, cu, table, pool, pool)
    with pytest.raises(ValueError, match="4-bit pools"):
        qa.qa_kvq_write(rows, rows, cu, table, pool[:, :100], pool[:, :100])
    with pytest.raises(ValueError, match="4-bit pools"):
        qa.qa_kvq_read(pool, pool[:2], table, cu, 4)
    with pytest.raises(TypeError, match="v must be a torch.Tensor"):
        qa.qa_kvq_write(rows, None, cu, table, pool, pool)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        qa.qa_rope_rows(rows, rows, lens)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        qa.qa_rope_rows(np.zeros((4, 8, 128)), rows, lens)
    with pytest.raises(ValueError, match="CUDA"):
        qa.qa_kvq_decode_attn(rows, pool, pool, table, lens)
    with pytest.raises(ValueError, match="3 dims"):
        qa.qa_kvq_decode_attn(rows[0], pool, pool, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        qa.qa_kvq_decode_step(rows, rows, rows, lens, lens, table, lens, pool, pool)


def test_code_places_cover_every_nibble_once():
    for is_k in (True, False):
        at, nib = _kvq.PLACES[is_k]
        assert sorted((2 * at + nib).ravel()) == list(range(2048))


def test_quantiser_definition():
    rng = np.random.default_rng(1)
    bits = wl.normal_bf16(rng, (50, 128))
    n, sm = _kvq.quantise(bits)
    x = wl.bf16_to_f64(bits).reshape(50, 4, 32)
    s, m = wl.bf16_to_f64(sm[..., 0]), wl.bf16_to_f64(sm[..., 1])
    back = m[..., None] + s[..., None] * n.reshape(50, 4, 32)
    # half a step of s, and s itself is within 2^-8 of range / 15: 15 codes of it add 15 * 2^-8 steps at the far end
    assert (np.abs(back - x) <= s[..., None] * (0.5 + 15 * 2.0 ** -8)).all()
    assert n.min() == 0 and n.max() == 15
    const = np.full((1, 128), 0x3F81, np.uint16)
    n, sm = _kvq.quantise(const)
    assert not n.any() and not sm[..., 0].any() and (sm[..., 1] == 0x3F81).all()


def test_put_and_read_rows():
    rng = np.random.default_rng(2)
    bits = wl.normal_bf16(rng, (37, 2, 128))
    table, pages = _kvq.page_table(rng, [50])
    for is_k in (True, False):
        pool = rng.integers(0, 256, size=(pages, 2 * 1280), dtype=np.uint8)
        _kvq.put_rows(pool, table[0], 13, bits, is_k)
        s, m, n = _kvq.rows(pool, table[0], 13, 37, is_k)
        codes, sm = _kvq.quantise(bits)
        np.testing.assert_array_equal(n, codes.transpose(1, 0, 2))
        np.testing.assert_array_equal(s[..., ::32], wl.bf16_to_f64(sm[..., 0]).transpose(1, 0, 2))
        np.testing.assert_array_equal(m[..., ::32], wl.bf16_to_f64(sm[..., 1]).transpose(1, 0, 2))
