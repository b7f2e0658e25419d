"""Copies of a key/value cache are caches of their own."""
import copy
import io
import pickle

import pytest
import torch

import test_kv_cache as kv


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def tensors(c):
    return c.k8, c.v8, c.k_scale, c.v_scale, c.table, c.spare, c.lens


def saved(c):
    f = io.BytesIO()
    torch.save(c, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


HOW = {"deepcopy": copy.deepcopy, "pickle": lambda c: pickle.loads(pickle.dumps(c)), "save": saved}


@pytest.mark.gpu
@pytest.mark.parametrize("how", HOW)
def test_a_copy_and_its_original_do_not_meet(lm, how):
    c = kv.filled(lm, 4, 90, 2, 64, 16, torch.float16, seed=1, layers=2)
    c.lens.fill_(20)
    d = HOW[how](c)
    r = kv.gen(1)
    k, q, parents = r(4, 7, 2, 64).half(), r(4, 1, 2, 64).half(), torch.tensor([[1, 0], [1, 1]], dtype=torch.int32, device="cuda")
    want = c.attend(1, q)
    assert torch.equal(d.attend(1, q), want)
    was = [t.clone() for t in tensors(c)]
    d.append(1, k, k)
    d.advance(7)
    d.reorder(parents)
    for a, b in zip(was, tensors(c)):
        assert torch.equal(a, b)
    assert not torch.equal(d.k8, c.k8) and not torch.equal(d.table, c.table) and d.lens.tolist() == [27] * 4
    c.append(1, k, k)
    c.advance(7)
    c.reorder(parents)
    for a, b in zip(tensors(c), tensors(d)):
        assert torch.equal(a, b)
    got = c.attend(1, q)
    del c  # the copy does not live on its original's memory
    torch.cuda.empty_cache()
    assert torch.equal(d.attend(1, q), got)


@pytest.mark.gpu
def test_a_shallow_copy_shares_the_tensors(lm):
    c = kv.filled(lm, 2, 64, 1, 64, 32, torch.bfloat16, seed=2)
    d = copy.copy(c)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(tensors(c), tensors(d)))
    k = kv.gen(2)(2, 5, 1, 64).bfloat16()
    d.append(0, k, k)
    d.advance(5)
    assert c.lens.tolist() == [5, 5] and torch.equal(c.read(0, 0, 5)[0], d.read(0, 0, 5)[0])


def test_no_address_is_copied():
    """Without a GPU: the state that copies are made of holds no packed pointers, and tensors off the GPU are refused."""
    from log_mel_spectrogram_gb300 import KvCache
    c = KvCache.__new__(KvCache)
    c.__dict__.update(_args=b"pointers", _head=(b"pointers", 0, 2), rows=1, heads=1, head_dim=32, layers=1, block=16, width=1,
                      blocks=2, max_tokens=16, dtype=torch.float16, _code=2, device=torch.device("cuda", 0))
    for name in ("_k8", "_v8", "_k_scale", "_v_scale", "_table", "_spare", "_lens"):
        setattr(c, name, torch.zeros(1))
    assert not any(isinstance(v, (bytes, tuple)) for v in c.__getstate__().values())
    for f in (copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        with pytest.raises(ValueError, match="CUDA"):
            f(c)
