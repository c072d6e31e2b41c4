"""The recurrent rule on wide batches of many tokens whose K and V differ, with either type and either gate,
against its plain 64-bit form: shapes whose columns do not fill a warp's 32. Tolerances of
test_gpu_recurrent."""
import pytest

from test_gpu_recurrent import BF, F32, _lib, call, check_o, check_state, make, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,V", [(128, 64), (64, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("gate_k", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay_first", [False, True])
def test_many_tokens_wide(K, V, gate_k, dtype, decay_first):
    # (4 x 152 blocks of 64 columns and more, a mean of 16 tokens; lengths even, odd, none and one)
    lens = [30, 2, 17, 0, 1, 46] * 16
    d = make(lens, 8, 4, K, V, dtype=dtype, gate_k=gate_k, seed=K + V)
    n = len(lens)
    slots_in = [-1 if i % 3 == 2 else d["order"][i] for i in range(n)]
    slots_out = [-7 if i % 5 == 4 else d["order"][n + i] for i in range(n)]
    after, err = call(d, slots_in, slots_out, decay_first=decay_first)
    assert err == (0, 0)
    o_ref, ref = reference(d, slots_in, slots_out, decay_first=decay_first)
    check_o(d, o_ref)
    check_state(d, after, ref, [x for x in slots_out if x >= 0])
