"""Host-side checks of the 4-bit cache's and the log probabilities' calls: every
call below is refused (or is a no-op) before any launch, so none needs a GPU."""
import ctypes

import pytest
import torch

from sparse_kv_verification_gb300 import build, native
from tests.test_abi_serving import FAKE, desc
from tests.test_native_serving import calls  # noqa: F401  (a recorder in the library's place)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.load()


def desc4(paged=False, base=FAKE, **kw):
    kv = native.DustinKV4()
    kv.data = base
    kv.stride_b, kv.stride_h, kv.stride_n = 2 * 4096 * 144, 4096 * 144, 144
    if paged:
        kv.page_table, kv.page_size, kv.pages_per_seq, kv.num_pages = FAKE, 16, 64, 128
    for name, value in kw.items():
        setattr(kv, name, value)
    return kv


def test_record_sizes(lib):
    size = lib.dustin_kv4_record_size
    assert size(64) == 80 and size(128) == 144 and size(96) == 0 and size(0) == 0


@pytest.mark.parametrize("name", ["write", "read"])
def test_write_and_read_refusals(lib, name):
    def call(layers=1, b=2, hkv=2, d=128, n=256, rows=32, kv=None, kv4=None, a=None, lens=None,
             null=False):
        kv, kv4 = kv or [desc(base=FAKE + 0x10000000)], kv4 or [desc4()]
        ka, k4 = (native.DustinKV * len(kv))(*kv), (native.DustinKV4 * len(kv4))(*kv4)
        pair = [ctypes.addressof(ka), ctypes.addressof(k4)]
        if null:
            pair = [None, pair[1]]
        if name == "read":
            pair = pair[::-1]
        return getattr(lib, "dustin_kv4_" + name)(layers, b, hkv, d, n, rows, *pair, a, lens, None)
    assert call(layers=-1) == 2 and call(b=-1) == 2 and call(hkv=0) == 2 and call(rows=-1) == 2
    assert call(n=-1) == 2 and call(d=96) == 3 and call(null=True) == 1
    assert call(a=FAKE + 2) == 5 and call(lens=FAKE + 1) == 5
    assert call(b=1 << 20, hkv=1 << 6, rows=1 << 6) == 2                  # 2^32 records
    assert call(kv=[desc(v=None)]) == 1 and call(kv=[desc(stride_n=100)]) == 2
    assert call(kv=[desc(True, base=FAKE + 0x10000000, pages_per_seq=1)]) == 2
    assert call(kv4=[desc4(data=None)]) == 1 and call(kv4=[desc4(base=FAKE + 8)]) == 5
    assert call(kv4=[desc4(stride_n=128)]) == 2 and call(kv4=[desc4(stride_h=-16)]) == 2
    assert call(kv4=[desc4(stride_n=152)]) == 5 and call(kv4=[desc4(stride_b=8)]) == 5
    assert call(kv4=[desc4(k_exp=65)]) == 2 and call(kv4=[desc4(v_exp=-65)]) == 2
    assert call(kv4=[desc4(True, page_size=24)]) == 3 and call(kv4=[desc4(True, num_pages=0)]) == 2
    assert call(kv4=[desc4(True, pages_per_seq=15)]) == 2                 # 240 of 256 positions
    shared = [dict(stride_h=0), dict(stride_b=0)]
    for s in shared:                                                      # rows on one another
        assert (call(kv4=[desc4(**s)]) == 2) if name == "write" else (call(kv=[desc(**s)]) == 2)
    if name == "read":
        assert call(rows=257) == 2                                        # k > n without idx
        assert call(n=0) == 2
    assert call(layers=0) == 0 and call(b=0) == 0 and call(rows=0, null=True) == 0


def test_attention_refusals(lib):
    def call(b=4, hq=8, hkv=2, d=128, w=4, n=256, k=256, q=FAKE, kv=desc4(), idx=None, k_len=None,
             win=None, scale=0.1, o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, flags=0):
        ref = lambda x: None if x is None else ctypes.byref(x)
        return lib.dustin_kv4_verify_attn(b, hq, hkv, d, w, n, k, q, ref(kv), idx, k_len, ref(win),
                                          scale, o, lse, ws, ws_bytes, flags, None)
    assert call(b=-1) == 2 and call(n=-1, k=0) == 2 and call(k=-1) == 2 and call(w=0) == 2
    assert call(hq=7) == 2 and call(d=96) == 3
    assert call(k=257) == 2                                               # more than there are
    assert call(n=1 << 28, k=(1 << 27) + 1) == 2 and call(b=(1 << 20) + 1, hq=1, hkv=1) == 2
    assert call(b=1 << 10, hkv=64, hq=64, n=1 << 27, k=1 << 27) == 2      # 32-bit work line
    assert call(q=None) == 1 and call(o=None) == 1 and call(lse=None) == 1 and call(kv=None) == 1
    assert call(q=FAKE + 8) == 5 and call(idx=FAKE + 2) == 5 and call(k_len=FAKE + 1) == 5
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(flags=2) == 1
    # scale * 2^k_exp within [2^-120, 2^126]; a call in range gets as far as its workspace.
    low, high = desc4(k_exp=-64), desc4(k_exp=64)
    assert call(scale=2.0 ** 127) == 2 and call(scale=1e20, kv=high) == 2
    assert call(scale=2.0 ** -121) == 2 and call(scale=2.0 ** -57, kv=low) == 2
    for kw in (dict(scale=2.0 ** 126), dict(scale=2.0 ** -120), dict(scale=2.0 ** 62, kv=high),
               dict(scale=2.0 ** -56, kv=low)):
        assert call(ws=None, **kw) == 4
    assert call(scale=2.0 ** 127, k=0, kv=None, ws=None) == 4                   # no cache, no such product
    assert call(kv=desc4(stride_n=100)) == 2 and call(kv=desc4(k_exp=-70)) == 2
    assert call(kv=desc4(True, pages_per_seq=15)) == 2 and call(kv=desc4(True, page_size=8)) == 3
    assert call(win=desc(True)) == 3 and call(win=desc(k=None)) == 1
    assert call(ws=None) == 4 and call(ws_bytes=1000) == 4 and call(ws=FAKE + 8) == 4
    assert "workspace" in lib.dustin_last_error().decode()
    assert call(b=0, q=None) == 0
    size = lib.dustin_kv4_verify_attn_workspace_size
    assert size(4, 8, 2, 128, 4, 256) > 0 and size(4, 8, 2, 128, 4, 0) > 0
    assert size(0, 8, 2, 128, 4, 256) == 0 and size(4, 8, 2, 96, 4, 256) == 0
    assert size(1 << 20, 64, 1, 128, 1, 16) == 0                          # past 2^35 bytes


def test_logprobs_refusals(lib):
    def call(b=2, w=3, vocab=100, dtype=0, x=FAKE, st=(300, 100), scale=1.0, rows=None, m=1,
             tokens=FAKE, lp=FAKE, ent=None, lse=None, top=2, ids=FAKE, best=FAKE):
        return lib.dustin_token_logprobs(b, w, vocab, dtype, x, *st, scale, rows, m, tokens, lp, ent,
                                         lse, top, ids, best, None)
    assert call(b=-1) == 2 and call(w=-1) == 2 and call(vocab=0) == 2
    assert call(vocab=(1 << 30) + 1) == 2 and call(b=1 << 20, w=1 << 8) == 2
    assert call(m=-1) == 2 and call(top=-1) == 2 and call(vocab=4, top=5) == 2
    assert call(m=513) == 3 and call(top=65) == 3
    assert call(dtype=2) == 1 and call(scale=0.0) == 1 and call(scale=float("nan")) == 1
    assert call(scale=float("inf")) == 1 and call(scale=1e31) == 1
    assert call(x=None) == 1 and call(tokens=None) == 1 and call(lp=None) == 1
    assert call(ids=None) == 1 and call(best=None) == 1
    assert call(st=(-1, 100)) == 2 and call(st=(300, -1)) == 2
    assert call(x=FAKE + 2) == 5 and call(dtype=1, x=FAKE + 1) == 5 and call(rows=FAKE + 2) == 5
    for a in ("tokens", "lp", "ent", "lse", "ids", "best"):
        assert call(**{a: FAKE + 2}) == 5
    assert call(b=0, x=None) == 0 and call(w=0, x=None) == 0


def test_binding_refusals(calls, monkeypatch):  # noqa: F811
    N = native
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    cache = u8(2, 2, 32, 144)
    with pytest.raises(ValueError, match="CUDA"):
        N.kv4_desc(cache)                                # on the CPU
    real = torch.Tensor.get_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0 if t.device.type == "cpu" else real(t))
    for bad in (cache.int(), cache[0], cache[..., ::2]):
        with pytest.raises(ValueError, match="uint8"):
            N.kv4_desc(bad)
    with pytest.raises(ValueError, match="page_table"):
        N.kv4_desc(cache, i32(2, 4).long())
    with pytest.raises(ValueError, match="contiguous"):
        N.kv4_desc(cache, i32(2, 8)[:, ::2])
    kv4, rows = N.kv4_desc(cache), N.kv_desc(bf(2, 2, 4, 128), bf(2, 2, 4, 128))
    with pytest.raises(ValueError, match="one src and one dst"):
        N.dustin_kv4_write([rows, rows], [kv4], 2, 2, 128, 32, 4)
    with pytest.raises(ValueError, match="start"):
        N.dustin_kv4_write([rows], [kv4], 2, 2, 128, 32, 4, start=i32(3))
    with pytest.raises(ValueError, match="idx"):
        N.dustin_kv4_read([kv4], [rows], 2, 2, 128, 32, 4, idx=i32(2, 5))
    q, o, lse = bf(2, 4, 3, 128), bf(2, 4, 3, 128), torch.zeros(2, 4, 3)
    attn = lambda q=q, o=o, lse=lse, **k: N.dustin_kv4_verify_attn(q, kv4, 2, 32, 32, 0.1, o, lse,
                                                                   u8(10), **k)
    for kw, what in ((dict(q=q.float()), "q must"), (dict(o=o[:, :2]), "o must"),
                     (dict(lse=lse.double()), "lse"), (dict(idx=i32(2, 31)), "idx"),
                     (dict(k_len=i32(1)), "k_len")):
        with pytest.raises(ValueError, match=what):
            attn(**kw)
    x = torch.zeros(2, 3, 50)
    lp = lambda x=x, tokens=i32(2, 3, 1), logprobs=torch.zeros(2, 3, 1), **k: \
        N.dustin_token_logprobs(x, tokens, logprobs, **k)
    for kw, what in ((dict(x=x.half()), "fp32 or bf16"), (dict(x=x[0]), "logits"),
                     (dict(x=torch.zeros(2, 3, 100)[..., ::2]), "contiguous"),
                     (dict(x=torch.zeros(2, 3, 1).expand(2, 3, 50)), "contiguous"),
                     (dict(logprobs=None), "come with"), (dict(top_ids=i32(2, 3, 4)), "come with"),
                     (dict(tokens=i32(2, 4, 1)), "tokens"), (dict(lse=torch.zeros(2)), "lse"),
                     (dict(entropy=torch.zeros(2, 3).double()), "entropy"),
                     (dict(n_rows=i32(3)), "n_rows")):
        with pytest.raises(ValueError, match=what):
            lp(**kw)
    assert not calls
    N.dustin_kv4_write([rows], [kv4], 2, 2, 128, 32, 4, start=i32(2), w_len=i32(2))
    N.dustin_kv4_read([kv4], [rows], 2, 2, 128, 32, 4)
    attn(idx=i32(2, 32), k_len=i32(2))
    lp(top_ids=i32(2, 3, 4), top_logprobs=torch.zeros(2, 3, 4), lse=torch.zeros(2, 3))
    N.dustin_token_logprobs(x, None, None, entropy=torch.zeros(2, 3))
    assert len(calls) == 5


def test_caches_of_two_devices_are_refused(calls):  # noqa: F811
    a, b = native.DustinKV4(), native.DustinKV4()
    a.index, b.index = 0, 1
    rows = native.DustinKV()
    with pytest.raises(ValueError, match="one device"):
        native.dustin_kv4_write([rows, rows], [a, b], 1, 1, 64, 4, 1)
    assert not calls


def test_attention_refuses_parts_longer_than_a_wait(lib):
    """Where a CTA has five units or more, the warp that deals them out waits for whole
    ones, at most 2^18 tiles of 128 positions."""
    def call(hkv, k, w=1):
        kv = desc4()
        return lib.dustin_kv4_verify_attn(1, hkv, hkv, 64, w, 1, k, FAKE, ctypes.byref(kv), FAKE, None,
                                          None, 0.1, FAKE, FAKE, None, 0, 0, None)
    size = lib.dustin_kv4_verify_attn_workspace_size
    assert call(760, 1 << 26) == 2 and call(257, (1 << 25) + 1) == 2 and call(3, 1 << 26, w=64 * 86) == 2
    assert size(1, 257, 257, 64, 1, 1 << 26) == 0 and size(257, 1, 1, 64, 1, 1 << 26) == 0
    for hkv, k, w in ((256, 1 << 26, 1), (760, 1 << 25, 1), (3, 1 << 26, 64 * 85)):
        assert call(hkv, k, w) == 4 and size(1, hkv, hkv, 64, w, k) > 0      # as far as the workspace
