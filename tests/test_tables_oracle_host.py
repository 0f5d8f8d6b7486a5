"""The block tables' oracle where the free pages run out, by hand."""

import oracle


def test_requests_behind_one_that_is_short():
    # five free pages: the first request needs ten and takes none, the others take one each, from the end
    cu, pos, slots, lens, left, table, status = oracle.block_tables_ref([160, 1, 16], [0, 0, 0], [3, 4, 5, 6, 7], 5, [[-1] * 10] * 3, 16, 180)
    assert cu == [0, 160, 161, 177] and lens == [0, 1, 16] and left == 3 and status == 32
    assert table[0] == [-1] * 10 and table[1][:2] == [7, -1] and table[2][:2] == [6, -1]
    assert slots[:160] == [-1] * 160 and slots[160] == 7 * 16 and slots[161:177] == [6 * 16 + i for i in range(16)]
    assert slots[177:] == [-1] * 3 and pos[161:177] == list(range(16))


def test_a_request_without_pages_or_tokens_is_not_short():
    _, _, _, lens, left, _, status = oracle.block_tables_ref([40, 3, 0], [0, 5, 20], [1], 1, [[-1] * 3, [9, -1, -1], [7, 8, -1]], 16, 50)
    assert lens == [0, 8, 20] and left == 1 and status == 32
