"""The Python binding's own refusals for the serving operators, on the CPU: the
library call is replaced by a recorder, so nothing is launched or read."""
import pytest
import torch

from sparse_kv_verification_gb300 import native as N


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(N, "_one_device", lambda *ts: 0)
    monkeypatch.setattr(N, "_run", lambda fn, index, stream, *args: made.append(args))
    monkeypatch.setattr(N, "load", lambda *a, **k: type("Lib", (), {"__getattr__": lambda s, n: n})())
    return made


def verify(p, q, b, w):
    N.dustin_verify_tokens(p, q, torch.zeros((b, w - 1), dtype=torch.int32), torch.zeros((b, w - 1)),
                           torch.zeros(b), torch.zeros((b, w), dtype=torch.int32),
                           torch.zeros(b, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabulary_rows_of_either_tensor_are_contiguous(calls, dtype):
    """Each side's entries lie one behind another, whatever the other side's
    do: an expanded (stride 0) row would be read past its storage."""
    b, w, vocab = 2, 3, 50
    p, q = torch.rand((b, w, vocab)).to(dtype), torch.rand((b, w - 1, vocab)).to(dtype)
    flat = lambda n: torch.tensor(1.0 / vocab, dtype=dtype).expand(b, n, vocab)
    spread = lambda n: torch.rand((b, n, 2 * vocab)).to(dtype)[:, :, ::2]
    for bad_p, bad_q in ((p, flat(w - 1)), (flat(w), q), (flat(w), flat(w - 1)), (p, spread(w - 1)),
                         (spread(w), q), (flat(w), None), (spread(w), None)):
        with pytest.raises(ValueError, match="contiguous"):
            verify(bad_p, bad_q, b, w)
    assert not calls
    # Rows may be shared, and cut out of longer ones.
    verify(p, q, b, w)
    verify(p[:1, :1].expand(b, w, vocab), q[:, :1].expand(b, w - 1, vocab), b, w)
    verify(torch.rand((b, w, 60)).to(dtype)[:, :, 7:57], None, b, w)
    verify(p[:, :, :1], q[:, :, :1].as_strided((b, w - 1, 1), (0, 0, 0)), b, w)   # one entry
    verify(p[:, :1], flat(0), b, 1)                                               # no draft rows
    assert len(calls) == 5
