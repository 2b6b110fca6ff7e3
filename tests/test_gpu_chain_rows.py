"""The decode chain with attention, where the rows' pages do not suffice: a row that the pass
does not serve keeps what it has cached, as the rows do that share its pages."""
import pytest
import torch

from nvfp4_sm_skinny_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, CONTEXT, PS = synth.HIDDEN, 40, 16


@pytest.mark.parametrize("captured", [False, True])
def test_rows_that_are_refused_or_wait_keep_their_tokens(captured):
    import nvfp4_sm_skinny_gb300 as sk
    from nvfp4_sm_skinny_gb300.chain import DecodeChain

    m = 5
    c = DecodeChain(layers=2, m=m, device=DEV, context=CONTEXT, kv_heads=2, page_size=PS)
    c.set_input(synth.normal_bf16((m, H), 1.0, 1).to(DEV), synth.normal_f32((m, H), 2).to(DEV))

    def want(*lens):
        c.want.copy_(torch.tensor(lens, dtype=torch.int32))

    for step in range(5):
        want(step + 1, 0, step + 1, step + 1, 0)
        c.forward()
    want(5, 0, 48, 20, 0)
    c.rows()
    # row 1 becomes a copy of row 0, row 4 of row 3: their last pages are shared
    sk.kv_fork(torch.tensor([-1, 0, -1, -1, 3], dtype=torch.int32, device=DEV), c.table, c.lens, c.refs, PS)
    # no page is free any more: held by somebody else
    c.refs.masked_fill_(c.refs == 0, 1)
    want(-1, -1, -1, -1, -1)
    run = c.capture().replay if captured else c.forward  # capture() runs a pass, of rows that wait
    lens = [5, 5, 48, 20, 20]
    saved, table = c.cache.clone(), c.table.clone()
    # rows 0 and 3 would have to leave the page that they share, row 2 is full, 1 and 4 wait
    want(6, -1, 49, 21, -1)
    c.set_input(synth.normal_bf16((m, H), 1.0, 3).to(DEV), synth.normal_f32((m, H), 4).to(DEV))
    run()
    torch.cuda.synchronize()
    assert c.row_status.tolist() == [1, 0, 2, 1, 0] and c.lens.tolist() == lens
    assert torch.equal(c.cache, saved) and torch.equal(c.table, table)
    # row 1 ends, so row 0 has its page for itself, and row 4 its last one; row 3 still shares its own
    want(-1, 0, -1, 10, -1)
    c.rows()
    saved = c.cache.clone()
    want(6, -1, -1, 11, 21)
    run()
    torch.cuda.synchronize()
    assert c.row_status.tolist() == [0, 0, 0, 1, 0] and c.lens.tolist() == [6, 0, 48, 10, 21]
    changed = (c.cache != saved).flatten(2).any(2).any(0).nonzero().flatten().tolist()
    assert sorted(changed) == sorted([int(c.table[0, 0]), int(c.table[4, 1])]) and sk.device_status() == 0
