"""4-bit KV cache without a GPU: the plain statement the GPU tests use, sizes,
struct layouts, and every refusal (all of them before any CUDA call)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

from tests import kv4_reference as ref


@pytest.fixture(scope="module")
def aq():
    from precision_attention_numerics_gb300 import _build
    _build.build()
    import precision_attention_numerics_gb300 as aq
    aq.load_library()
    return aq


def test_reference_rounds_to_the_formats():
    v = torch.arange(-700, 701, dtype=torch.float64) / 100
    near = ref.e2m1(v)
    grid = torch.cat((-ref.E2M1.flip(0), ref.E2M1))
    assert torch.equal((near - v).abs(), (grid[None, :] - v.clamp(-6, 6)[:, None]).abs().amin(1) + (v.abs() - 6).clamp(min=0))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 7.0])
    assert ref.e2m1(ties).tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.0, -4.0, 6.0]
    x = torch.cat((torch.logspace(-12, 8.8, 4001, base=2.0), torch.arange(0, 448, 0.25)))
    assert torch.equal(ref.e4m3(x), x.to(torch.float8_e4m3fn).double())
    assert ref.e4m3(torch.tensor([449.0, 1e30])).tolist() == [448.0, 448.0]


def test_reference_rotation_keeps_products():
    g = torch.Generator().manual_seed(1)
    a, b = torch.randn(5, 128, generator=g), torch.randn(5, 128, generator=g)
    signs = torch.randint(0, 2, (128,), generator=g) * 2 - 1
    # fp32 butterflies: 8 roundings of at most 2^-24 of the row's norm each side
    err = (ref.rotate(a, signs).double() * ref.rotate(b, signs).double()).sum(-1) - (a.double() * b.double()).sum(-1)
    assert (err.abs() <= 16 * 2.0 ** -24 * 2 * a.norm(dim=-1) * b.norm(dim=-1)).all()


def test_cache_bytes(aq):
    mk = lambda **k: aq.AttnqKv4Cache(**{**dict(num_pages=10, page_tokens=64, Hkv=8, d=128), **k})
    assert aq.attnq_kv4_cache_bytes(mk()) == 10 * 64 * 8 * 144
    assert aq.attnq_kv4_cache_bytes(mk(num_pages=1 << 20)) == (1 << 20) * 64 * 8 * 144
    for bad in (dict(num_pages=0), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=512), dict(Hkv=0),
                dict(d=96), dict(flags=4)):
        assert aq.attnq_kv4_cache_bytes(mk(**bad)) == 0
        assert aq.attnq_kv4_attn_workspace(mk(**bad), 1, 1, 8, 1) == 0
    assert aq.attnq_kv4_attn_workspace(mk(), 1, 1, 9, 1) == 0  # 9 query heads on 8
    assert aq.attnq_kv4_attn_workspace(mk(), 65536, 1, 8, 1) == 0
    assert aq.attnq_kv4_attn_workspace(mk(), 2, 4, 32, 5) > 0
    assert aq.attnq_kv4_evict_workspace(mk(), 2, 4, 0) == 0
    assert aq.attnq_kv4_evict_workspace(mk(), 2, 4, 16) > 0


def test_struct_layouts_match_the_header(aq, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text(
        "#include <stdio.h>\n#include \"attnq.h\"\nint main(void) { printf(\"%zu %zu %zu %zu %zu %zu %zu\\n\","
        " sizeof(attnq_kv4_cache), offsetof(attnq_kv4_cache, signs), offsetof(attnq_kv4_cache, pages),"
        " sizeof(attnq_kv4_seqs), offsetof(attnq_kv4_seqs, new_lens), sizeof(attnq_rows),"
        " offsetof(attnq_rows, stride_t)); return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(root, "include"), "-I", cuda_inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    from precision_attention_numerics_gb300 import binding as b
    assert got == [C.sizeof(b._Kv4Cache), b._Kv4Cache.signs.offset, b._Kv4Cache.pages.offset, C.sizeof(b._Kv4Seqs),
                   b._Kv4Seqs.new_lens.offset, C.sizeof(b._Rows), b._Rows.stride_t.offset]
    # the packed forms that calls pass are the same bytes
    assert b._pack_kv4_cache(1, 2, 3, 4, 5, 6, 7, 8, 9) == bytes(b._Kv4Cache(1, 2, 3, 4, 5, 6, 7, 8, 9))
    assert b._pack_kv4_seqs(1, 2, 3, 4, 5) == bytes(b._Kv4Seqs(1, 2, 3, 4, 5))
    assert b._pack_rows(1, 2, 3, 4, -5) == bytes(b._Rows(1, 2, 3, 4, -5))


FAKE = 1 << 20  # never dereferenced: every call below is refused on the host


def _cache(aq, **k):
    from precision_attention_numerics_gb300 import binding as b
    f = dict(num_pages=8, page_tokens=16, Hkv=2, d=64, flags=0, signs=None, k_scale=None, v_scale=None, pages=FAKE)
    f.update(k)
    return b._Kv4Cache(*f.values())


def _seqs(aq, **k):
    from precision_attention_numerics_gb300 import binding as b
    f = dict(B=2, max_pages=4, table=FAKE, lens=FAKE + 256, new_lens=None)
    f.update(k)
    return b._Kv4Seqs(*f.values())


def _rows(aq, H=2, T=3, d=64, **k):
    from precision_attention_numerics_gb300 import binding as b
    f = dict(data=FAKE, dtype=1, sb=H * T * d, sh=T * d, st=d)
    f.update(k)
    return b._Rows(*f.values())


BAD_CACHES = [(dict(pages=None), 1), (dict(pages=FAKE + 8), 1), (dict(num_pages=0), 1), (dict(Hkv=0), 1),
              (dict(flags=1), 1), (dict(flags=1, signs=FAKE + 8), 1), (dict(flags=8), 1), (dict(d=96), 2), (dict(page_tokens=24), 2),
              (dict(k_scale=FAKE + 2), 1)]
BAD_SEQS = [(dict(B=0), 1), (dict(B=40000), 2), (dict(max_pages=0), 1), (dict(max_pages=1 << 25), 2),
            (dict(table=None), 1), (dict(lens=None), 1), (dict(table=FAKE + 1), 1), (dict(new_lens=FAKE + 2), 1)]
BAD_ROWS = [dict(data=None), dict(data=FAKE + 8), dict(dtype=2), dict(st=68), dict(sh=1 << 60), dict(sb=-64)]
OVERLAPPING = [dict(st=0), dict(st=32), dict(sh=64), dict(sb=0), dict(sb=192)]


def _call_append(L, c, s, T, k, v, mean=None):
    return L.attnq_kv4_append(C.byref(c), C.byref(s), T, C.byref(k), C.byref(v), mean, None)


def test_append_and_read_refusals(aq):
    L = aq.load_library()
    for bad, rc in BAD_CACHES:
        assert _call_append(L, _cache(aq, **bad), _seqs(aq), 3, _rows(aq), _rows(aq)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert _call_append(L, _cache(aq), _seqs(aq, **bad), 3, _rows(aq), _rows(aq)) == rc, bad
    for bad in BAD_ROWS:
        assert _call_append(L, _cache(aq), _seqs(aq), 3, _rows(aq, **bad), _rows(aq)) == 1, bad
        assert _call_append(L, _cache(aq), _seqs(aq), 3, _rows(aq), _rows(aq, **bad)) == 1, bad
    assert _call_append(L, _cache(aq), _seqs(aq), 0, _rows(aq), _rows(aq)) == 1
    assert _call_append(L, _cache(aq), _seqs(aq), 3, _rows(aq, dtype=0), _rows(aq)) == 1  # K and V of two types
    assert _call_append(L, _cache(aq), _seqs(aq), 3, _rows(aq), _rows(aq), FAKE) == 1  # a mean without the flag
    assert _call_append(L, _cache(aq, flags=2), _seqs(aq), 3, _rows(aq), _rows(aq)) == 1  # the flag without a mean
    for bad in BAD_ROWS + OVERLAPPING:
        rc = L.attnq_kv4_read(C.byref(_cache(aq)), C.byref(_seqs(aq)), 3, C.byref(_rows(aq, data=FAKE + (1 << 16))),
                              C.byref(_rows(aq, **bad)), None)
        assert rc == 1, bad
    same = _rows(aq)  # both outputs in one place
    assert L.attnq_kv4_read(C.byref(_cache(aq)), C.byref(_seqs(aq)), 3, C.byref(same), C.byref(same), None) == 1


def test_attention_refusals(aq):
    L = aq.load_library()

    def call(c=None, s=None, T=3, Hq=4, q=None, o=None, scale=0.125, causal=1, lse=None, ai=None, ao=None, ws=FAKE,
             nb=1 << 40):
        q, o = q or _rows(aq, H=4), o or _rows(aq, H=4, data=FAKE + (1 << 16))
        return L.attnq_kv4_attn(C.byref(c or _cache(aq)), C.byref(s or _seqs(aq)), T, Hq, C.byref(q), C.byref(o),
                                C.c_float(scale), causal, lse, ai, ao, ws, nb, None)
    for bad, rc in BAD_CACHES:
        assert call(c=_cache(aq, **bad)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert call(s=_seqs(aq, **bad)) == rc, bad
    for bad in BAD_ROWS:
        assert call(q=_rows(aq, H=4, **bad)) == 1, bad
    for bad in BAD_ROWS + OVERLAPPING:
        assert call(o=_rows(aq, H=4, **bad)) == 1, bad
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == 1
    assert call(Hq=3) == 1 and call(Hq=0) == 1 and call(causal=2) == 1 and call(T=0) == 1
    assert call(Hq=1 << 28) == 2
    assert call(ai=FAKE) == 1  # weights in without weights out
    assert call(lse=FAKE + 1) == 1 and call(ao=FAKE + 2) == 1
    assert call(ws=None) == 1 and call(ws=FAKE + 128) == 1 and call(nb=0) == 1
    assert call(o=_rows(aq, H=4)) == 1  # over the queries


def test_evict_refusals(aq):
    L = aq.load_library()

    def call(c=None, s=None, acc=FAKE, budget=32, sink=4, recent=8, table=FAKE + 512, pages=2, lens=FAKE + 1024,
             kept=FAKE + 2048, out=None, ws=FAKE, nb=1 << 40):
        return L.attnq_kv4_evict(C.byref(c or _cache(aq)), C.byref(s or _seqs(aq)), acc, budget, sink, recent, table,
                                 pages, lens, kept, out, ws, nb, None)
    for bad, rc in BAD_CACHES:
        assert call(c=_cache(aq, **bad)) == rc, bad
    for bad, rc in BAD_SEQS:
        assert call(s=_seqs(aq, **bad)) == rc, bad
    for bad in (dict(acc=None), dict(table=None), dict(lens=None), dict(kept=None), dict(budget=0), dict(pages=0),
                dict(sink=-1), dict(recent=-1), dict(sink=30), dict(budget=33), dict(lens=FAKE + 256),
                dict(out=FAKE), dict(table=FAKE), dict(ws=None), dict(nb=0), dict(kept=FAKE + 2),
                dict(kept=FAKE + 1024)):
        assert call(**bad) == 1, bad
    assert call(pages=1 << 25) == 2


def test_no_calls_in_the_kernel_that_moves_registers(tmp_path):
    """kv4_prefill.cu's warps run on different register budgets (setmaxnreg). A device
    function that the compiler does not inline is built for the launch's budget, so
    calling it from a warp that has given registers away is undefined (seen once as a
    kernel that did not end): the compiler must report no function but the kernels."""
    from precision_attention_numerics_gb300 import _build
    r = subprocess.run([_build._nvcc(), *_build.NVCC_FLAGS, "-Xptxas", "-v", "-c",
                        os.path.join(_build.CSRC, "kv4_prefill.cu"), "-o", str(tmp_path / "x.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    functions = [l for l in r.stderr.splitlines() if "Function properties for" in l]
    assert functions and all("k_kv4_prefill" in f or "k_kv4_join" in f for f in functions), functions


def test_attention_workspace_grows_with_the_call(aq):
    """A buffer for the largest call serves every smaller one, and what a call must have is that less the scores."""
    mk = lambda **k: aq.AttnqKv4Cache(**{**dict(num_pages=10, page_tokens=64, Hkv=8, d=128), **k})
    for cache in (mk(), mk(Hkv=1, d=64), mk(Hkv=3, page_tokens=16)):
        for G in (1, 3, 4, 7):
            size = lambda B, pages, T, G=G: aq.attnq_kv4_attn_workspace(cache, B, pages, G * cache.Hkv, T)
            for B, pages, T in ((8, 512, 1), (16, 512, 1), (1, 8, 5), (2, 40, 9), (300, 4, 2)):
                last = 0
                for t in (1, 2, 3, 4, 5, 6, 8, 9, 16, 17, 24, 25, 32, 33, 64, 65, 100, 257, 1024):
                    assert size(B, pages, t) >= last, (B, pages, t, G)
                    last = size(B, pages, t)
                last = 0
                for b in (1, 2, 3, 5, 8, 16, 17, 40, 100, 300, 1000, 5000):
                    assert size(b, pages, T) >= last, (b, pages, T, G)
                    last = size(b, pages, T)
                last = 0
                for n in (1, 2, 3, 7, 8, 20, 64, 100, 512, 513, 1024, 2048, 5000, 100000):
                    assert size(B, n, T) >= last, (B, n, T, G)
                    last = size(B, n, T)
            last = 0
            for g in range(1, 40):
                assert size(8, 512, 1, G=g) >= last
                last = size(8, 512, 1, G=g)
    # the least that a call takes, as attnq.h states it: a byte less is refused (on the host)
    L = aq.load_library()
    for B, pages, Hq, T in ((2, 4, 4, 1), (2, 4, 4, 3), (2, 1 << 20, 4, 1), (2, 4, 64, 40)):
        c, s = _cache(aq), _seqs(aq, B=B, max_pages=pages)
        q, o = _rows(aq, H=Hq, T=T), _rows(aq, H=Hq, T=T, data=FAKE + (1 << 24))
        rows = T * Hq // 2
        tail = min(64 << 20, B * 2 * pages * 16 * (16 if rows <= 4 else 32 * -(-rows // 8)))
        least = L.attnq_kv4_attn_workspace(C.byref(c), B, pages, Hq, T) - -(-tail // 256) * 256
        assert least > 0
        assert L.attnq_kv4_attn(C.byref(c), C.byref(s), T, Hq, C.byref(q), C.byref(o), C.c_float(0.125), 1, None, None,
                                None, FAKE, least - 1, None) == 1


def test_sizes_past_32_bits_are_not_cut_off(aq):
    mk = lambda **k: aq.AttnqKv4Cache(**{**dict(num_pages=10, page_tokens=64, Hkv=8, d=128), **k})
    w = 1 << 32
    for bad in (dict(num_pages=w + 10), dict(page_tokens=w + 64), dict(Hkv=w + 8), dict(d=w + 128)):
        assert aq.attnq_kv4_cache_bytes(mk(**bad)) == 0
        assert aq.attnq_kv4_attn_workspace(mk(**bad), 1, 1, 8, 1) == 0
        assert aq.attnq_kv4_evict_workspace(mk(**bad), 1, 1, 1) == 0
        with pytest.raises(aq.AttnqError):
            aq.alloc_kv4_cache(**{**dict(num_pages=10, page_tokens=64, Hkv=8, d=128), **bad}, device="cpu")
    for i in range(4):
        sizes = [1, 1, 8, 1]
        assert aq.attnq_kv4_attn_workspace(mk(), *sizes) > 0
        sizes[i] += w
        assert aq.attnq_kv4_attn_workspace(mk(), *sizes) == 0
    for i in range(3):
        sizes = [1, 1, 1]
        sizes[i] += w
        assert aq.attnq_kv4_evict_workspace(mk(), *sizes) == 0
