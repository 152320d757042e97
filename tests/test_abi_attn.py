"""Host-side checks of include/kda_attn.h (no GPU): every declared function is exported, and bad
arguments are refused before any device work, by the C entries and by the bindings."""
import os
import re

import pytest
import torch

import gated_delta_rule_78_amd as kda
from gated_delta_rule_78_amd import attn
from gated_delta_rule_78_amd.attn import HeadRopeDesc, KvAppendDesc, PagedAttnDesc, PageStrides, RowStrides

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first
GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_78_amd import build
        build.build()
    return attn._library()


def p(i, off=0):
    return FAKE + i * 64 * GB + off


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kda_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kda_[a-z_]+)\s*\(", text))
    assert len(names) == 6
    for n in names:
        assert hasattr(lib, n), n


# ---- norm and rotation --------------------------------------------------------------------------

def rows(H, T, d):
    return RowStrides(H * T * d, T * d, d)


def rdesc(B=2, Hq=4, Hk=2, T=10, d=64, rot=64, q=None, k=None, qo=None, ko=None, dq=None, dk=None, dtype=1, inter=0, norm=1,
          eps=1e-6, scale=1.0):
    r = lambda s, H: s if s is not None else rows(H, T, d)
    return HeadRopeDesc(B, Hq, Hk, T, d, rot, r(q, Hq), r(k, Hk), r(qo, Hq), r(ko, Hk), r(dq, Hq), r(dk, Hk), dtype, inter, norm,
                        eps, scale)


BAD_ROPE = (dict(B=0), dict(Hq=-1), dict(Hq=0, Hk=0), dict(T=-1), dict(d=0), dict(d=63, rot=0), dict(rot=63), dict(rot=66),
            dict(rot=-2), dict(dtype=2), dict(inter=2), dict(norm=-1), dict(eps=0.0), dict(eps=float("nan")),
            dict(eps=float("inf")), dict(scale=float("nan")), dict(scale=float("inf")))


def rfwd(lib, d, q=p(0), k=p(1), wq=None, wk=None, f=p(2), pos=None, qo=p(3), ko=p(4)):
    return lib.kda_head_rope_fwd(d, q, k, wq, wk, f, pos, qo, ko, None)


def test_rope_fwd_refusals(lib):
    assert rfwd(lib, None) == INVALID
    for bad in BAD_ROPE:
        assert rfwd(lib, rdesc(**bad)) == INVALID, bad
    assert rfwd(lib, rdesc(d=1026, rot=0), f=None) == UNSUPPORTED
    assert rfwd(lib, rdesc(Hq=5000)) == UNSUPPORTED
    assert rfwd(lib, rdesc(B=1 << 16, T=1 << 15)) == UNSUPPORTED
    for k in ("q", "k", "qo", "ko", "f"):
        assert rfwd(lib, rdesc(), **{k: None}) == INVALID, k
    assert rfwd(lib, rdesc(rot=0)) == INVALID                                 # frequencies without rotation
    assert rfwd(lib, rdesc(norm=0), wq=p(5)) == INVALID                       # a weight without norm
    for k in ("q", "k", "qo", "ko", "f", "wq", "wk", "pos"):
        assert rfwd(lib, rdesc(), **{k: p(6, 1)}) == INVALID, k               # off its element
    assert rfwd(lib, rdesc(), qo=p(0)) == INVALID                             # not in place
    assert rfwd(lib, rdesc(), qo=p(4, 128)) == INVALID                        # outputs overlap
    assert rfwd(lib, rdesc(), ko=p(2, 16)) == INVALID                         # the frequencies inside an output
    assert rfwd(lib, rdesc(q=RowStrides(-1, 640, 64))) == INVALID             # negative stride
    assert rfwd(lib, rdesc(q=RowStrides(1 << 62, 640, 64))) == INVALID        # past any address
    assert rfwd(lib, rdesc(q=RowStrides(0, 1 << 33, 64))) == UNSUPPORTED      # head strides have 32 bits
    for bad in (RowStrides(2560, 0, 64), RowStrides(2560, 640, 32), RowStrides(0, 640, 64)):
        assert rfwd(lib, rdesc(qo=bad)) == INVALID                            # rows of an output share elements
    assert rfwd(lib, rdesc(T=0), q=None, k=None, qo=None, ko=None) == OK      # nothing to do


def rbwd(lib, d, q=p(0), k=p(1), wq=None, wk=None, f=p(2), pos=None, zq=p(3), zk=p(4), dq=p(5), dk=p(6), dwq=None, dwk=None,
         ws=p(7), ws_bytes=1 << 30):
    return lib.kda_head_rope_bwd(d, q, k, wq, wk, f, pos, zq, zk, dq, dk, dwq, dwk, ws, ws_bytes, None)


def test_rope_bwd_refusals(lib):
    assert rbwd(lib, None) == INVALID
    for bad in BAD_ROPE:
        assert rbwd(lib, rdesc(**bad)) == INVALID, bad
    for k in ("q", "k", "zq", "zk", "dq", "dk", "f"):
        assert rbwd(lib, rdesc(), **{k: None}) == INVALID, k
    assert rbwd(lib, rdesc(norm=0), dwq=p(8)) == INVALID
    assert rbwd(lib, rdesc(Hq=0), dwq=p(8)) == INVALID                        # a gradient for no heads
    for k in ("q", "k", "zq", "zk", "dq", "dk", "dwq", "dwk"):
        assert rbwd(lib, rdesc(), **{k: p(9, 1)}) == INVALID, k
    assert rbwd(lib, rdesc(), dq=p(0)) == INVALID
    assert rbwd(lib, rdesc(), dq=p(3)) == INVALID
    assert rbwd(lib, rdesc(), dwq=p(8), dwk=p(8)) == INVALID
    need = lib.kda_head_rope_bwd_workspace_bytes(rdesc())
    assert need > 0 and lib.kda_head_rope_bwd_workspace_bytes(rdesc(norm=0)) == 0
    assert lib.kda_head_rope_bwd_workspace_bytes(rdesc(T=0)) == 0 and lib.kda_head_rope_bwd_workspace_bytes(None) == 0
    assert rbwd(lib, rdesc(), dwq=p(8), ws=None) == WORKSPACE
    assert rbwd(lib, rdesc(), dwq=p(8), ws_bytes=need - 1) == WORKSPACE
    assert rbwd(lib, rdesc(), dwq=p(8), ws=p(7, 8)) == INVALID
    assert rbwd(lib, rdesc(), dwq=p(8), ws=p(0)) == INVALID
    assert rbwd(lib, rdesc(T=0), q=None, k=None, zq=None, zk=None, dq=None, dk=None) == OK


# ---- append -------------------------------------------------------------------------------------

def pages(H, page, d):
    return PageStrides(H * page * d, page * d, d)


def adesc(N=3, Hq=4, Hk=2, T=5, dk=64, dv=32, rot=64, pg=20, page=16, most=4, stride=4, dtype=1, packed=0, inter=0, norm=1,
          eps=1e-6, scale=1.0, kc=None, vc=None, qo=None):
    return KvAppendDesc(N, Hq, Hk, T, dk, dv, rot, pg, page, most, stride, rows(Hq, T, dk), rows(Hk, T, dk), rows(Hk, T, dv),
                        qo or rows(Hq, T, dk), kc or pages(Hk, page, dk), vc or pages(Hk, page, dv), dtype, packed, inter, norm,
                        eps, scale)


def app(lib, d, q=p(0), k=p(1), v=p(2), wq=None, wk=None, f=p(3), cu=None, lens=p(4), table=p(5), qo=p(6), kc=p(7), vc=p(8)):
    return lib.kda_kv_append(d, q, k, v, wq, wk, f, cu, lens, table, qo, kc, vc, None)


def test_append_refusals(lib):
    assert app(lib, None) == INVALID
    for bad in (dict(N=0), dict(Hq=-1), dict(Hk=0), dict(T=-1), dict(dk=0), dict(dk=63, rot=0), dict(dv=0), dict(rot=65),
                dict(pg=0), dict(page=0), dict(most=0), dict(stride=3), dict(dtype=3), dict(packed=2), dict(inter=2),
                dict(norm=2), dict(eps=0.0), dict(scale=float("nan"))):
        assert app(lib, adesc(**bad)) == INVALID, bad
    for bad in (dict(dk=2048, rot=0), dict(dv=1025), dict(page=(1 << 20) + 1), dict(most=1 << 28, stride=1 << 28), dict(pg=1 << 31),
                dict(N=1 << 30, T=4)):
        assert app(lib, adesc(**bad), f=None if bad.get("rot") == 0 else p(3)) == UNSUPPORTED, bad
    for k in ("q", "k", "v", "lens", "table", "qo", "kc", "vc", "f"):
        assert app(lib, adesc(), **{k: None}) == INVALID, k
    assert app(lib, adesc(), cu=p(9)) == INVALID                              # cu_seqlens only with packed
    assert app(lib, adesc(packed=1)) == INVALID
    for k in ("q", "k", "v", "lens", "table", "qo", "kc", "vc", "f", "wq", "wk"):
        assert app(lib, adesc(), **{k: p(10, 1)}) == INVALID, k
    assert app(lib, adesc(), kc=p(1)) == INVALID
    assert app(lib, adesc(), qo=p(7, 64)) == INVALID
    assert app(lib, adesc(), vc=p(7)) == INVALID                              # the same pages twice
    assert app(lib, adesc(), vc=p(7, 64)) == INVALID
    assert app(lib, adesc(), table=p(8, 16)) == INVALID
    assert app(lib, adesc(kc=PageStrides(2048, 1024, 32))) == INVALID         # a cache's rows share elements
    assert app(lib, adesc(qo=RowStrides(0, 320, 64))) == INVALID
    assert app(lib, adesc(T=0), q=None, k=None, v=None, qo=None, kc=None, vc=None, lens=None, table=None) == OK


@pytest.mark.parametrize("strides, gap, ok", [
    ((8192, 1024, 64), 4096, True),      # [pages, 2, Hk, page, d]: values behind a page's keys
    ((4096, 2048, 64), 1024, True),      # [pages, Hk, 2, page, d]
    ((4096, 2048, 128), 64, True),       # [pages, Hk, page, 2, d]
    ((4096, 2048, 128), 32, False),      # rows overlap by half
    ((4096, 1024, 64), 2048, True),      # values in the second half of a page's stride
    ((4096, 1024, 64), 1024, False),     # the second head's keys
    ((4096, 1024, 64), 4096, False),     # the next page's keys
    ((6000, 1024, 64), 2048, True),
    ((6000, 1024, 64), 5000, False),     # runs into the next page
])
def test_caches_may_interleave_but_not_share(lib, strides, gap, ok):
    d = adesc(dk=64, dv=64, kc=PageStrides(*strides), vc=PageStrides(*strides))
    # without a device a call that passes validation answers KDA_ERR_HIP; with one it is not made
    if ok and torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    assert (app(lib, d, kc=p(7), vc=p(7, 2 * gap)) != INVALID) == ok


# ---- attention ----------------------------------------------------------------------------------

def tdesc(N=3, Hq=4, Hk=2, T=5, dk=64, dv=64, pg=20, page=16, most=4, stride=4, window=0, packed=0, scale=0.125, q=None, o=None,
          kc=None, vc=None):
    return PagedAttnDesc(N, Hq, Hk, T, dk, dv, pg, page, most, stride, window, q or rows(Hq, T, dk), o or rows(Hq, T, dv),
                         kc or pages(Hk, page, dk), vc or pages(Hk, page, dv), packed, scale)


def att(lib, d, q=p(0), kc=p(1), vc=p(2), cu=None, lens=p(3), table=p(4), o=p(5), lse=None, ws=p(6), ws_bytes=1 << 34):
    return lib.kda_paged_attn(d, q, kc, vc, cu, lens, table, o, lse, ws, ws_bytes, None)


def test_attn_refusals(lib):
    assert att(lib, None) == INVALID
    for bad in (dict(N=0), dict(Hq=0), dict(Hk=0), dict(Hq=5), dict(T=-1), dict(pg=0), dict(page=0), dict(most=0), dict(stride=3),
                dict(window=-1), dict(packed=2), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert att(lib, tdesc(**bad)) == INVALID, bad
    for bad in (dict(dk=32), dict(dk=192), dict(dv=256), dict(page=24), dict(page=1 << 21), dict(Hq=1024, Hk=1024), dict(pg=1 << 31),
                dict(most=1 << 28, stride=1 << 28), dict(T=1 << 30)):
        assert att(lib, tdesc(**bad)) == UNSUPPORTED, bad
    for k in ("q", "kc", "vc", "lens", "table", "o"):
        assert att(lib, tdesc(), **{k: None}) == INVALID, k
        assert att(lib, tdesc(), **{k: p(7, 1)}) == INVALID, k
    for k in ("q", "kc", "vc", "o"):
        assert att(lib, tdesc(), **{k: p(7, 8)}) == INVALID, k                # off 16 bytes
    assert att(lib, tdesc(), lse=p(7, 2)) == INVALID
    assert att(lib, tdesc(), cu=p(7)) == INVALID
    assert att(lib, tdesc(packed=1)) == INVALID
    assert att(lib, tdesc(q=RowStrides(1280, 324, 64))) == UNSUPPORTED        # rows off 8 elements
    assert att(lib, tdesc(kc=PageStrides(4096, 1024, 68))) == UNSUPPORTED
    assert att(lib, tdesc(kc=PageStrides(1 << 32, 1024, 64))) == UNSUPPORTED  # a page past 32 bits
    assert att(lib, tdesc(page=1 << 20, most=1, kc=PageStrides(1 << 30, 1 << 29, 1032))) == UNSUPPORTED
    assert att(lib, tdesc(o=RowStrides(1280, 0, 64))) == INVALID
    assert att(lib, tdesc(), o=p(0)) == INVALID
    assert att(lib, tdesc(), o=p(1, 1024)) == INVALID
    assert att(lib, tdesc(), lse=p(5)) == INVALID
    need = lib.kda_paged_attn_workspace_bytes(tdesc())
    assert need > 0 and lib.kda_paged_attn_workspace_bytes(tdesc(T=0)) == 0 and lib.kda_paged_attn_workspace_bytes(None) == 0
    assert att(lib, tdesc(), ws=None) == WORKSPACE
    assert att(lib, tdesc(), ws_bytes=need - 1) == WORKSPACE
    assert att(lib, tdesc(), ws=p(6, 8)) == INVALID
    assert att(lib, tdesc(), ws=p(1)) == INVALID
    assert att(lib, tdesc(T=0), q=None, kc=None, vc=None, o=None, lens=None, table=None, ws=None) == OK


# ---- the bindings refuse on the host what the C call cannot see ----

def test_bindings_refuse():
    z = lambda *s: torch.zeros(*s)
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, k, f = z(2, 4, 5, 8), z(2, 2, 5, 8), z(4)
    with pytest.raises(ValueError, match="GPU"):
        kda.head_rope_fwd(q, k, f)
    with pytest.raises(ValueError, match="one of q and k"):
        kda.head_rope_fwd(None, None, f)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.head_rope_fwd(q.half(), k.half(), f)
    with pytest.raises(ValueError, match=r"\[H,T,d\]"):
        kda.head_rope_fwd(q[0, 0], None, f)
    with pytest.raises(ValueError, match="k must be"):
        kda.head_rope_fwd(q, k[:, :, :4], f)
    with pytest.raises(ValueError, match="k must be"):
        kda.head_rope_fwd(q, k.bfloat16(), f)
    with pytest.raises(ValueError, match="q must be"):
        kda.head_rope_fwd(z(2, 4, 5, 16)[..., ::2], k, f)
    with pytest.raises(ValueError, match="inv_freq"):
        kda.head_rope_fwd(q, k, f.double())
    with pytest.raises(ValueError, match="inv_freq"):
        kda.head_rope_fwd(q, k, z(2, 2))
    with pytest.raises(ValueError, match="positions"):
        kda.head_rope_fwd(q, k, f, i(5))
    with pytest.raises(ValueError, match="positions"):
        kda.head_rope_fwd(q, k, f, i(2, 5).long())
    with pytest.raises(ValueError, match="q_weight goes"):
        kda.head_rope_fwd(q, k, f, q_weight=z(8), norm=False)
    with pytest.raises(ValueError, match="k_weight"):
        kda.head_rope_fwd(q, k, f, k_weight=z(9))
    kc, vc, table, lens = b(3, 2, 16, 8), b(3, 2, 16, 6), i(2, 4), i(2)
    v = z(2, 2, 5, 6)
    call = lambda **kw: kda.kv_append(*[kw.get(n, d) for n, d in (("q", q), ("k", k), ("v", v), ("kc", kc), ("vc", vc), ("table", table),
                                                                  ("lens", lens), ("f", f))],
                                      **{n: x for n, x in kw.items() if n in ("cu_seqlens", "q_weight", "norm")})
    with pytest.raises(ValueError, match="GPU"):
        call()
    for bad, what in ((dict(k=k.half(), q=q.half(), v=v.half()), "unsupported dtype"), (dict(v=z(2, 2, 4, 6)), "v must be"),
                      (dict(q=z(2, 4, 4, 8)), "q must be"), (dict(kc=z(3, 2, 16, 8)), "k_cache must be"),
                      (dict(kc=b(3, 1, 16, 8)), "k_cache must be"), (dict(vc=b(4, 2, 16, 6)), "v_cache must be"),
                      (dict(vc=b(3, 2, 16, 12)[..., ::2]), "v_cache must be"), (dict(kc=b(2, 16, 8)), "k_cache must be"),
                      (dict(table=i(3, 4)), "block_table"), (dict(table=i(2, 4).long()), "block_table"), (dict(lens=i(3)), "kv_lens"),
                      (dict(f=z(4).double()), "inv_freq"), (dict(cu_seqlens=i(3)), r"\[H,T,d\]"),
                      (dict(q_weight=z(8), norm=False), "q_weight goes")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    qb, kc, vc = b(2, 4, 5, 64), b(3, 2, 16, 64), b(3, 2, 16, 64)
    with pytest.raises(ValueError, match="GPU"):
        kda.paged_attn(qb, kc, vc, table, lens)
    for args, what in (((qb.float(), kc, vc, table, lens), "q must be"), ((qb, kc[..., :32], vc, table, lens), "k_cache must be"),
                       ((qb, kc, vc.float(), table, lens), "v_cache must be"), ((qb, kc, vc[0], table, lens), "must be"),
                       ((qb, kc, vc, table[:1], lens), "block_table"), ((qb, kc, vc, table, lens.long()), "kv_lens"),
                       ((qb[0], kc, vc, table, lens), r"\[H,T,d\]")):
        with pytest.raises(ValueError, match=what):
            kda.paged_attn(*args)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.paged_attn(qb[0], kc, vc, table, lens, cu_seqlens=i(3).long())
    with pytest.raises(ValueError, match="o must be"):
        kda.paged_attn(qb, kc, vc, table, lens, o=b(2, 4, 5, 32))
    with pytest.raises(ValueError, match="lse must be"):
        kda.paged_attn(qb, kc, vc, table, lens, lse=z(2, 4, 6))



# ---- calls past what a launch, an index or a scan of the lengths can hold ----

def test_limits(lib):
    big = (1 << 31) - 1
    one = dict(B=1, Hq=1, Hk=0, T=big, d=2, rot=2)
    assert rfwd(lib, rdesc(**one), k=None, ko=None) == UNSUPPORTED            # 2^27 workgroups
    assert rbwd(lib, rdesc(**one), k=None, zk=None, dk=None) == UNSUPPORTED
    assert rfwd(lib, rdesc(Hq=4097, q=RowStrides(0, 0, 0)), ko=p(9)) == UNSUPPORTED
    assert rfwd(lib, rdesc(q=RowStrides(0, 1 << 32, 64))) == UNSUPPORTED
    a = adesc(N=1, Hq=0, Hk=1, T=big, dk=2, dv=1, rot=2, most=1, stride=1)
    assert app(lib, a, q=None, qo=None) == UNSUPPORTED
    for bad in (dict(N=65537), dict(pg=1, most=(1 << 26) + 1, stride=1 << 27), dict(N=1, Hq=8, Hk=8, T=1 << 28), dict(N=2, T=1 << 30)):
        d = tdesc(**bad)
        assert att(lib, d, o=p(30)) == UNSUPPORTED and lib.kda_paged_attn_workspace_bytes(d) == 0, bad
    assert lib.kda_paged_attn_workspace_bytes(tdesc(N=65536)) > 0
    assert lib.kda_paged_attn_workspace_bytes(tdesc(most=1 << 26, stride=1 << 26)) > 0
