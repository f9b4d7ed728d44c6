"""Host-side checks of the serving operators: every call below is refused (or
is a no-op) before any launch, so none needs a GPU."""
import ctypes

import pytest

from sparse_kv_verification_gb300 import build, native

FAKE = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def desc(paged=False, base=FAKE, **kw):
    kv = native.DustinKV()
    kv.k = base
    kv.v = base + 0x100000
    kv.stride_b, kv.stride_h, kv.stride_n = 4096 * 128, 512 * 128, 128
    if paged:
        kv.page_table, kv.page_size, kv.pages_per_seq, kv.num_pages = FAKE, 16, 64, 128
    for name, value in kw.items():
        setattr(kv, name, value)
    return kv


def test_verify_tokens_refusals(lib):
    def call(b=2, w=4, vocab=100, dtype=0, p=FAKE, st=(400, 100), q=FAKE, sd=(300, 100), draft=FAKE,
             ua=FAKE, us=FAKE, tok=FAKE, acc=FAKE):
        return lib.dustin_verify_tokens(b, w, vocab, dtype, p, *st, q, *sd, draft, None, ua, us,
                                        tok, acc, None)
    assert call(b=-1) == 2 and call(w=0) == 2 and call(vocab=0) == 2
    assert call(dtype=2) == 1
    assert call(p=None) == 1 and call(us=None) == 1 and call(tok=None) == 1 and call(acc=None) == 1
    assert call(draft=None) == 1 and call(ua=None) == 1
    assert call(st=(-1, 100)) == 2 and call(sd=(300, -1)) == 2
    assert call(p=FAKE + 2) == 5 and call(dtype=1, p=FAKE + 1) == 5 and call(tok=FAKE + 2) == 5
    assert call(b=0, p=None) == 0


def test_compact_refusals(lib):
    def call(layers=1, b=2, hkv=2, d=128, n=256, k=32, src=None, dst=None, idx=FAKE, k_len=None):
        src = src or [desc()]
        dst = dst or [desc(base=FAKE + 0x1000000)]
        sa, da = (native.DustinKV * len(src))(*src), (native.DustinKV * len(dst))(*dst)
        return lib.dustin_kv_compact(layers, b, hkv, d, n, k, ctypes.addressof(sa),
                                     ctypes.addressof(da), idx, k_len, None)
    assert call(layers=-1) == 2 and call(b=-1) == 2 and call(hkv=0) == 2 and call(k=-1) == 2
    assert call(d=96) == 3
    assert call(idx=None) == 1 and call(idx=FAKE + 2) == 5 and call(k_len=FAKE + 1) == 5
    assert call(src=[desc(v=None)]) == 1 and call(dst=[desc(stride_n=100)]) == 2
    assert call(src=[desc(stride_h=4)]) == 5
    assert call(src=[desc(True, pages_per_seq=8)]) == 2           # 128 positions hold no n = 256
    assert call(dst=[desc(True, pages_per_seq=1)]) == 2           # nor 16 a k of 32
    assert call(src=[desc()], dst=[desc()], n=16, k=32) == 2      # in place, k > n
    assert call(src=[desc()], dst=[desc(v=FAKE)]) == 1            # K in place, V not
    assert call(src=[desc()], dst=[desc(stride_b=8)]) == 1        # one cache in two layouts
    two = [desc(), desc(True)]
    assert call(layers=2, src=two, dst=[desc(base=FAKE + 0x1000000)] * 2) == 1
    assert call(layers=0) == 0 and call(b=0) == 0 and call(k=0, idx=None) == 0


def test_fork_and_resize_refusals(lib):
    def fork(n=4, pp=8, page=16, pages=64, forks=2, parent=FAKE, child=FAKE, table=FAKE, ln=FAKE,
             rc=FAKE):
        return lib.dustin_kv_fork(n, pp, page, pages, forks, parent, child, table, ln, rc, None)

    def resize(n=4, pp=8, page=16, pages=64, m=2, seqs=FAKE, new=FAKE, table=FAKE, ln=FAKE, rc=FAKE,
               copies=FAKE, layers=0, hkv=2, d=128, kv=None):
        arr = (native.DustinKV * 1)(kv or desc(True, num_pages=64))
        return lib.dustin_kv_resize(n, pp, page, pages, m, seqs, new, table, ln, rc, copies, layers,
                                    hkv, d, ctypes.addressof(arr), None)
    for call in (fork, resize):
        assert call(n=0) == 2 and call(pp=0) == 2 and call(pages=0) == 2
        assert call(page=8) == 3 and call(page=24) == 3 and call(pages=(1 << 22) + 1) == 3
        assert call(pp=1 << 28) == 2 and call(n=1 << 30, pp=4) == 2
        assert call(table=None) == 1 and call(ln=None) == 1 and call(rc=FAKE + 2) == 5
    assert fork(forks=-1) == 2 and fork(parent=None) == 1 and fork(child=FAKE + 1) == 5
    assert fork(forks=0, table=None) == 0
    assert resize(m=-1) == 2 and resize(m=1025) == 3 and resize(layers=-1) == 2
    assert resize(seqs=None) == 1 and resize(copies=None) == 1 and resize(new=FAKE + 2) == 5
    assert resize(layers=1, hkv=0) == 2 and resize(layers=1, d=80) == 3
    assert resize(layers=1, kv=desc()) == 1                       # not paged
    assert resize(layers=1, kv=desc(True, num_pages=32)) == 1     # another pool
    assert resize(layers=1, kv=desc(True, num_pages=64, v=None)) == 1
    assert resize(m=0, table=None) == 0


def test_prefix_attention_refusals(lib):
    def call(b=4, groups=2, hq=8, hkv=2, d=128, w=4, n_p=256, n_o=64, q=FAKE, prefix=desc(),
             own=desc(), plen=None, olen=None, win=None, scale=0.1, o=FAKE, lse=FAKE, ws=FAKE,
             ws_bytes=1 << 40, flags=0):
        ref = lambda kv: None if kv is None else ctypes.byref(kv)
        return lib.dustin_prefix_verify_attn(b, groups, hq, hkv, d, w, n_p, n_o, q, ref(prefix), plen,
                                             ref(own), olen, ref(win), scale, o, lse, ws, ws_bytes,
                                             flags, None)
    assert call(groups=3) == 2 and call(groups=0) == 2 and call(b=-2) == 2
    assert call(n_p=-1) == 2 and call(n_o=-1) == 2 and call(w=0) == 2 and call(hq=7) == 2
    assert call(d=96) == 3
    assert call(n_p=1 << 30, hq=512, b=400) == 2                # 32-bit work line
    assert call(q=None) == 1 and call(o=None) == 1 and call(lse=None) == 1
    assert call(q=FAKE + 8) == 5 and call(plen=FAKE + 2) == 5 and call(olen=FAKE + 1) == 5
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(flags=2) == 1
    assert call(prefix=None) == 1 and call(own=None) == 1
    assert call(prefix=desc(v=None)) == 1 and call(own=desc(stride_n=100)) == 2
    assert call(prefix=desc(True, pages_per_seq=15)) == 2
    assert call(own=desc(True, page_size=24)) == 3
    assert call(win=desc(True)) == 3 and call(win=desc(k=None)) == 1
    assert call(ws=None) == 4 and call(ws_bytes=1000) == 4 and call(ws=FAKE + 8) == 4
    assert "workspace" in lib.dustin_last_error().decode()
    assert call(b=0, q=None) == 0
    size = lib.dustin_prefix_verify_attn_workspace_size
    assert size(4, 2, 8, 2, 128, 4, 256, 64) > 0
    assert size(4, 3, 8, 2, 128, 4, 256, 64) == 0 and size(0, 1, 8, 2, 128, 4, 256, 64) == 0


def test_refusals_of_shared_rows_and_sizes(lib):
    def compact(src, dst, b=2, hkv=2, k=32):
        return lib.dustin_kv_compact(1, b, hkv, 128, 256, k, ctypes.byref(src), ctypes.byref(dst),
                                     FAKE, None, None)
    other = FAKE + 0x1000000
    for name in ("stride_b", "stride_h", "stride_n"):
        assert compact(desc(), desc(base=other, **{name: 0})) == 2
    assert compact(desc(True), desc(True, base=other, stride_b=0)) == 2
    assert compact(desc(True), desc(True, pages_per_seq=32)) == 1     # in place, another table
    assert lib.dustin_kv_fork(2, (1 << 26) + 1, 16, 64, 1, FAKE, FAKE, FAKE, FAKE, FAKE, None) == 2

    size = lib.dustin_prefix_verify_attn_workspace_size
    assert size(1, 1, 1, 1, 64, 1, 1 << 27, 0) > 0
    assert size(1, 1, 1, 1, 64, 1, (1 << 27) + 1, 0) == 0
    assert size(1, 1, 1, 1, 64, 1, 0, (1 << 27) + 1) == 0
    assert size((1 << 20) + 1, 1, 1, 1, 64, 1, 0, 16) == 0
    # 2^20 sequences of 128 rows: a place of 64 KB per part of one
    assert size(1 << 20, 1, 128, 1, 128, 1, 0, 16) == 0


def test_compact_refuses_lists_past_its_32_bit_counts(lib):
    src, dst = desc(), desc(base=FAKE + 0x1000000)
    for k in ((1 << 30) + 1, 0x7fffffff):
        assert lib.dustin_kv_compact(1, 2, 2, 128, 256, k, ctypes.byref(src), ctypes.byref(dst), FAKE,
                                     None, None) == 2
    assert "too large" in lib.dustin_last_error().decode()
