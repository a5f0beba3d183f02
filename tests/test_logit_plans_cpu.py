"""What the plans over logits refuse before anything is launched, with stand-ins for CUDA
tensors: they have sizes, strides and a device, but no memory."""
import pytest
import torch

from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class OnDevice(torch.Tensor):
    """A tensor without memory that says it is on CUDA device 0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))
    data_ptr = lambda self: 0x10000  # noqa: E731


def fake(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnDevice)


BIG = 2**32 + 5  # a C int of the same bits is 5


def plans(lead, V, K):
    """Every plan over logits [*lead, V] and a teacher's K entries, on stand-ins."""
    x = fake(*lead, V, dtype=torch.bfloat16)
    i32 = torch.int32
    f, two, ids, val = fake(*lead), fake(*lead, 2), fake(*lead, K, dtype=i32), fake(*lead, K)
    grad = fake(*lead, V, dtype=torch.bfloat16)
    yield lambda: kb.LogprobsPlan(x, fake(*lead, dtype=i32), logprob_out=f, entropy_out=f, stats_out=two,
                                  top_ids_out=fake(*lead, 0, dtype=i32), top_logprobs_out=fake(*lead, 0), stream=0)
    yield lambda: kb.LogprobsBackwardPlan(x, None, two, f, grad_entropy=f, dlogits=grad, stream=0)
    yield lambda: kb.DistillPlan(x, ids, val, loss_out=f, stats_out=two, stream=0)
    yield lambda: kb.DistillBackwardPlan(x, ids, val, two, dlogits=grad, stream=0)
    yield lambda: kb.DistillStepPlan(x, ids, val, loss_out=f, stats_out=two, dlogits=grad, stream=0)


@pytest.mark.parametrize("lead,V", [((1,), BIG), ((BIG,), 8), ((2**16, 2**16), 8), ((1,), 2**31), ((2**31,), 8)])
def test_sizes_past_32_bits_are_refused(lead, V):
    for make in plans(lead, V, 4):
        with pytest.raises(ValueError, match="32 bits"):
            make()


def test_teacher_entries_and_kinds_past_32_bits_are_refused():
    for make in list(plans((1,), 8, 2**32 + 4))[2:]:
        with pytest.raises(ValueError, match="32 bits"):
            make()
    x, ids, val = fake(2, 8), fake(2, 4, dtype=torch.int32), fake(2, 4)
    with pytest.raises(ValueError, match="32 bits"):
        kb.DistillPlan(x, ids, val, kind=2**32, loss_out=fake(2), stats_out=fake(2, 2), stream=0)


def test_the_largest_sizes_reach_the_library():
    """Rows of 2^30 logits make a plan; the library itself refuses one more."""
    for make in plans((2,), 2**30, 4):
        make()
    for make in plans((2,), 2**30 + 1, 4):
        with pytest.raises(kb.KdaError, match="V must lie in"):
            make()()


def test_a_plan_is_launched_on_the_device_of_its_tensors(monkeypatch):
    """Pointers of one device are not handed to a kernel of another: neither when the plan is made,
    which takes the current stream, nor at a later call.  (No rows: nothing is launched.)"""
    current = [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    made = [make() for make in plans((0,), 8, 4)]
    for plan in made:
        plan()
    current[0] = 1
    for plan, make in zip(made, plans((0,), 8, 4)):
        with pytest.raises(RuntimeError, match="current device"):
            plan()
        with pytest.raises(RuntimeError, match="current device"):
            make()
    current[0] = 0
    for plan in made:
        plan()
