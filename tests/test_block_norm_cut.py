"""How block_norm_backward cuts its rows, at sizes that no test allocates: the host's arithmetic alone,
without a GPU. The kernel writes dx and dh with 32-bit offsets inside a block of rows and reads vectors
with 32-bit offsets too."""
import pytest

I32 = 2 ** 31 - 1
MAX_ROW = {False: 65536, True: 32768}  # columns of a row of 131072 bytes: bf16, fp32


@pytest.fixture(scope="module")
def bsq():
    import __graft_entry__

    __graft_entry__.build()
    import block_scaled_precision_bsq_gb300 as b

    return b


COLS = [1, 2, 7, 8, 64, 100, 255, 256, 768, 1001, 4088, 4089, 4090, 4095, 4096, 4097, 4100, 8192, 9001, 16384, 20000,
        32761, 32768, 32769, 40000, 65521, 65529, 65530, 65535, 65536]
ROWS = [1, 8, 300, 51200, 290000, 295000, 300000, 700000, 5000000, I32]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vectors", [False, True])
@pytest.mark.parametrize("sms", [1, 132, 152])
def test_offsets_inside_a_block_fit_32_bits(bsq, f32, vectors, sms):
    flags = bsq.FLAG_SRC_F32 if f32 else 0
    for cols in COLS:
        if cols > MAX_ROW[f32]:
            continue
        for rows in ROWS:
            for widest in (cols, 2 * cols + 8, 1 << 20, I32):
                c = bsq.bsq_test_norm_cut(flags, rows, cols, 1, widest, vectors, sms)
                at = (cols, rows, widest, c)
                assert c.rows_per_block >= 1 and (c.blocks - 1) * c.rows_per_block < rows <= c.blocks * c.rows_per_block, at
                assert c.rows_per_block % (c.classes * c.teams) == 0, at
                # a thread's offset runs up to six steps past the block's rows before its last value is dropped
                around = 6 * c.classes * c.teams
                assert (c.rows_per_block + around) * cols <= I32, at
                assert not c.vectors or (c.rows_per_block + around) * max(cols, widest) <= I32, at
                assert vectors or not c.vectors, at
                # the partial sums of every block and class, of both norms
                assert c.workspace >= (2 * c.blocks * c.classes + c.classes) * 2 * cols * 4, at
                assert c.blocks * c.classes * c.cluster <= I32, at  # CTAs of the launch


def test_usual_sizes_take_one_block_an_sm(bsq):
    for rows, cols, blocks in ((14336, 768, 150), (51200, 1024, 151), (16384, 8192, 76)):
        c = bsq.bsq_test_norm_cut(0, rows, cols)
        assert c.vectors and abs(c.blocks - blocks) <= 2, c


def test_refusals(bsq):
    for bad, code in ((dict(rows=0, cols=64), bsq.ERR_ARG), (dict(rows=4, cols=0), bsq.ERR_ARG),
                      (dict(rows=4, cols=65537), bsq.ERR_SHAPE), (dict(rows=1 << 31, cols=64), bsq.ERR_SHAPE),
                      (dict(rows=4, cols=64, gate_groups=3), bsq.ERR_SHAPE), (dict(rows=4, cols=64, widest=-1), bsq.ERR_ARG),
                      (dict(rows=4, cols=64, num_sms=0), bsq.ERR_ARG)):
        with pytest.raises(bsq.BsqError) as e:
            bsq.bsq_test_norm_cut(0, **bad)
        assert e.value.code == code, bad


@pytest.mark.parametrize("f32", [False, True])
def test_no_row_takes_more_ctas_than_a_cluster_has(bsq, f32):
    """Rows that start inside 16-byte vectors cover up to a vector more: 65530 bf16 columns and more would
    take 17 CTAs by vectors, and are read element by element. All other widths stay with vectors."""
    flags = bsq.FLAG_SRC_F32 if f32 else 0
    vec, most = (4 if f32 else 8), MAX_ROW[f32]
    for cols in list(range(1, most + 1, 97)) + list(range(most - 40, most + 1)) + [4089, 4090, 4095, 4096, 4097]:
        for vectors in (False, True):
            c = bsq.bsq_test_norm_cut(flags, 1000, cols, vectors=vectors)
            assert 1 <= c.cluster <= 16 and c.warps * c.teams <= 16, (cols, c)
            # every column has a thread: 8 elements a thread, a row's first vector up to vec - 1 elements before it
            cover = cols + (vec - 1 if c.classes > 1 else 0)
            assert c.cluster * c.warps * 256 >= cover, (cols, c)
            assert c.vectors == (vectors and (f32 or cols <= 65529 or cols == 65536)), (cols, c)


@pytest.mark.parametrize("cols", [1001, 1020, 1022, 1023, 9001])
@pytest.mark.parametrize("group_rows", [1, 2, 3, 4, 7, 8, 16])
def test_workspace_of_many_gates_is_no_multiple_of_their_gradient(bsq, cols, group_rows):
    """A gate row's sums (two of dgate's size) have a slot for each alignment class, two or no more than the gate
    has rows, and one for each block that it is cut into."""
    groups = 6400
    rows = groups * group_rows
    for flags, vec in ((0, 8), (bsq.FLAG_SRC_F32, 4)):
        c = bsq.bsq_test_norm_cut(flags, rows, cols, groups)
        dgate = groups * cols * 4
        blocks = 152 * 2 * cols * 4 * 3
        slots = max(2, min(group_rows, vec))
        assert c.classes <= slots and c.workspace <= 2 * dgate * slots + blocks, c
    # a few gates keep to vectors: their slots are few
    assert bsq.bsq_test_norm_cut(0, 5 * group_rows, cols, 5).vectors
