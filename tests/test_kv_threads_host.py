"""Two threads on one object: the library reads each call's own arguments.  No GPU: stand-ins take the library's place."""
import threading

import pytest
import torch

from test_kv_host import q8  # noqa: F401

HEADS, DIM = 2, 64


@pytest.fixture
def host(q8, monkeypatch):  # noqa: F811
    """The binding with tensors of the host, whose device is -1."""
    from q8_matrix_vector_gb300 import kv, rotary

    for module in (kv, rotary):
        monkeypatch.setattr(module, "_current", lambda: -1)
        monkeypatch.setattr(module, "_stream", lambda device: 0)
    return kv, rotary


class Late:
    """An entry point that reads its arguments when as many callers as there are have come."""

    def __init__(self, struct, callers=2):
        self.struct, self.barrier, self.got = struct, threading.Barrier(callers, timeout=20), {}

    def __call__(self, *args):
        at = next(a for a in args if isinstance(a, bytes))
        self.barrier.wait()
        self.got[threading.get_ident()] = self.struct.from_buffer_copy(at)
        self.barrier.wait()
        return 0


def run(calls):
    """The calls' results, each by a thread of its own; by thread's number, what the entry point read."""
    out, errors = {}, []

    def go(i, call):
        try:
            out[i] = (threading.get_ident(), call())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=(i, c)) for i, c in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    return [out[i] for i in range(len(calls))]


def plan(cls, **fields):
    p = cls.__new__(cls)
    p.__dict__.update(device=-1, _where=torch.device("cpu"), _h=None, **fields)
    return p


def cache_of(kv, prefix="q8kv_cache"):
    c = kv.Cache.__new__(kv.Cache)
    c.__dict__.update(device=-1, _tail=(HEADS, DIM), _ref=object(), heads=HEADS, head_dim=DIM)
    return c


def test_rotation_and_write(host):
    kv, rotary = host
    late = Late(rotary.WriteArgs)
    r = plan(rotary.Rotary, head_dim=DIM, rotary_dim=DIM, _fused={"kvrope_write_q8": late})
    tensors = [dict(q=torch.zeros(n, 4, DIM), k=torch.zeros(n, HEADS, DIM), v=torch.zeros(n, HEADS, DIM),
                    positions=torch.zeros(n, dtype=torch.int64), slots=torch.zeros(n, dtype=torch.int64)) for n in (3, 5)]
    done = run([lambda t=t: r.write(cache_of(kv), *t.values()) for t in tensors])
    for (who, out), t in zip(done, tensors):
        a = late.got[who]
        assert (a.q, a.k, a.v, a.positions, a.slots, a.n) == (*(t[n].data_ptr() for n in ("q", "k", "v", "positions", "slots")), len(t["q"]))
        assert a.out == out.data_ptr()


def test_attention(host):
    kv, _ = host
    late = Late(kv.AttendArgs)
    p = plan(kv.TreeAttention, heads=4, kv_heads=HEADS, _tail=(4, DIM), _packed=(4 * DIM, DIM), _scale=0.5, _fn=late)
    tensors = [(torch.zeros(n, 4, DIM), torch.zeros(n, 7, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)) for n in (1, 2)]
    done = run([lambda t=t: p(t[0], cache_of(kv), t[1], t[2]) for t in tensors])
    for (who, out), (q, table, lengths) in zip(done, tensors):
        a = late.got[who]
        assert (a.q, a.table, a.lengths, a.out, a.requests) == (q.data_ptr(), table.data_ptr(), lengths.data_ptr(), out.data_ptr(), len(q))


def test_verification(host):
    kv, _ = host
    late = Late(kv.VerifyArgs)
    p = plan(kv.TreeVerify, vocab=8, max_requests=1, _fn=late, _tail=(8,))
    tensors = [(torch.zeros(n, 8), *(torch.zeros(n, dtype=torch.int32) for _ in range(2)), torch.zeros(n)) for n in (3, 4)]
    done = run([lambda t=t: p(*t) for t in tensors])
    for (who, out), t in zip(done, tensors):
        a = late.got[who]
        assert (a.logits, a.tokens, a.parents, a.uniforms, a.rows) == (*(x.data_ptr() for x in t), len(t[0]))
        assert (a.path, a.count, a.next_token) == tuple(x.data_ptr() for x in out)
