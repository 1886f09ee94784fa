"""What the binding of the decode-side operators does with arguments that are
no tensors, raise, or leave rows of a new output without a value, and with its
outputs' memory."""
import pytest
import torch

import bit_weight_only_int4_amd as q4
from tests.gpu_util import need_gpu
from tests.test_serve_abi import binding_args, i32


@pytest.mark.parametrize("op", ["kv_append", "attention"])
def test_new_tokens_without_a_sequence_are_refused(op):
    """Their rows of a new output would hold whatever its memory held."""
    none = dict(page_table=torch.zeros((0, 2), dtype=torch.int32), cu_new=i32(0), lengths=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="sequence"):
        getattr(q4, op)(**binding_args(op, **none))


def test_a_bound_that_leaves_rows_of_a_new_output_out_is_refused():
    # 3 new tokens of one sequence
    with pytest.raises(ValueError, match="max_new"):
        q4.attention(**binding_args("attention", max_new=2))
    for kw in (dict(max_new=3), dict(max_new=2, out=torch.zeros((3, 4, 64)))):
        with pytest.raises(ValueError, match="must be a device tensor"):
            q4.attention(**binding_args("attention", **kw))


@pytest.mark.parametrize("op,name", [("kv_append", "k"), ("attention", "q"), ("kv_dequant", "k_cache"), ("token_logprobs", "logits"),
                                     ("token_logprobs_backward", "logits")])
@pytest.mark.parametrize("value", [[1.0], None, 3])
def test_a_first_argument_that_is_no_tensor(op, name, value):
    with pytest.raises(ValueError, match=f"{name} must be a tensor"):
        getattr(q4, op)(**binding_args(op, **{name: value}))


class Raises:
    def __bool__(self):
        raise KeyError("neither")


def test_an_argument_whose_truth_raises():
    with pytest.raises(KeyError, match="neither"):
        q4.kv_append(**binding_args("kv_append", interleaved=Raises()))


def own_memory(tensors):
    """No two share storage or a version counter."""
    assert len({t.untyped_storage().data_ptr() for t in tensors}) == len(tensors)
    assert all(t._base is None and t.storage_offset() == 0 for t in tensors)
    for i, t in enumerate(tensors):
        before = [x._version for x in tensors]
        t.add_(1)
        assert [x._version - v for x, v in zip(tensors, before)] == [j == i for j in range(len(tensors))]


@pytest.mark.gpu
def test_outputs_are_tensors_of_their_own():
    """An in-place change of one does not touch the others, nor what autograd
    saved of them, and none keeps another's memory."""
    need_gpu()
    for rows in (3, 400):
        r = q4.token_logprobs(torch.randn((rows, 3000), device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda"), top_k=4)
        own_memory(list(r))
    weight = torch.ones(400, device="cuda", requires_grad=True)
    loss = (r.logprob * weight).sum()  # saves logprob
    r.entropy.mul_(2)
    loss.backward()
    assert torch.equal(weight.grad, r.logprob)
    own_memory(list(q4.kv_dequant(*q4.new_cache(3, 2, 64, 16))))
