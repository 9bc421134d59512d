"""What the paged cache's, the attention's and the verification's calls refuse,
and their size functions: all on the host, before any device work (no GPU is
needed; addresses are made up)."""

import pytest

from test_abi_block import A, ALIGN, BF16, BIG, F16, F32, I8, INVALID, WORKSPACE, change, refuse


def test_page_sizes(q4lib):
    size = q4lib.q4_kv_page_size
    assert size(64, 8, 128, F16) == 64 * 8 * 128 * 2 * 2
    assert size(64, 8, 128, BF16) == size(64, 8, 128, F16)
    # codes, and two fp32 scales a token and head
    assert size(64, 8, 128, I8) == 64 * 8 * (128 * 2 + 8)
    # dims in whole chunks of 64
    assert size(16, 2, 72, F16) == 16 * 2 * 128 * 2 * 2
    for bad in ((8, 8, 128, F16), (48, 8, 128, F16), (2048, 8, 128, F16), (64, 0, 128, F16), (64, 8, 12, F16), (64, 8, 0, F16),
                (64, 8, 264, F16), (64, 8, 128, F32), (64, 8, 128, 9), (-64, 8, 128, F16)):
        assert size(*bad) == 0


def test_attention_workspace(q4lib):
    size = q4lib.q4_attention_workspace_size
    last = 0
    for rows in (1, 4, 5, 8, 9, 16, 17, 64, 1000, 100000):   # it does not fall as rows grow
        need = size(rows, 1, 32, 8, 128)
        assert need >= last and need % 4 == 0
        last = need
    for bad in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1025, 32, 8, 128), (1, 1, 30, 8, 128), (1, 1, 32, 8, 260),
                (1, 1, 32, 8, 100), (1 << 30, 1, 32, 8, 128), (-1, 1, 32, 8, 128), (1, 1, 0, 8, 128), (1, 1, 32, 0, 128)):
        assert size(*bad) == 0


# pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt, lens, starts, n_seq, K, ldk, V, ldv, type, rows
WRITE = [A, 10, 64, 2, 64, F16, A, 4, A, A, 2, A, 128, A, 128, F32, 3]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=0), INVALID), (dict(_1=1 << 31), INVALID), (dict(_2=24), INVALID), (dict(_3=0), INVALID),
    (dict(_4=60), INVALID), (dict(_4=512, _12=BIG, _14=BIG), INVALID), (dict(_5=F32), INVALID), (dict(_6=0), INVALID),
    (dict(_7=0), INVALID), (dict(_8=0), INVALID), (dict(_9=0), INVALID), (dict(_10=-1), INVALID), (dict(_10=1025), INVALID),
    (dict(_11=0), INVALID), (dict(_12=127), INVALID), (dict(_13=0), INVALID), (dict(_14=127), INVALID), (dict(_15=I8), INVALID),
    (dict(_16=-1), INVALID), (dict(_16=1 << 30), INVALID),
    (dict(_0=A + 8), ALIGN), (dict(_6=A + 2), ALIGN), (dict(_8=A + 2), ALIGN), (dict(_9=A + 2), ALIGN), (dict(_11=A + 2), ALIGN),
    (dict(_13=A + 2), ALIGN), (dict(_13=A + 1, _15=BF16), ALIGN),
])
def test_cache_write(q4lib, at, code):
    refuse(q4lib, "q4_kv_write", change(WRITE, **at), code)


# K, ldk, V, ldv, type, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt, first, starts, n_seq, rows
READ = [A, 128, A, 128, F32, A, 10, 64, 2, 64, I8, A, 4, A, A, 2, 3]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=127), INVALID), (dict(_2=0), INVALID), (dict(_3=127), INVALID), (dict(_4=I8), INVALID),
    (dict(_5=0), INVALID), (dict(_6=0), INVALID), (dict(_7=0), INVALID), (dict(_8=-1), INVALID), (dict(_9=4), INVALID),
    (dict(_10=F32), INVALID), (dict(_11=0), INVALID), (dict(_12=0), INVALID), (dict(_14=0), INVALID), (dict(_15=1025), INVALID),
    (dict(_16=-1), INVALID),
    (dict(_0=A + 2), ALIGN), (dict(_2=A + 2), ALIGN), (dict(_5=A + 4), ALIGN), (dict(_11=A + 1), ALIGN), (dict(_13=A + 2), ALIGN),
    (dict(_14=A + 2), ALIGN),
])
def test_cache_read(q4lib, at, code):
    refuse(q4lib, "q4_kv_read", change(READ, **at), code)


# O, ldo, Q, ldq, type, heads, scale, window, pages, n_pages, page_tokens, kv_heads, d, ctype, table, ldt, lens,
# starts, n_seq, rows, max_new, workspace, bytes
ATTEND = [A, 256, A, 256, F16, 4, 0.125, 0, A, 10, 64, 2, 64, F16, A, 4, A, A, 2, 3, 2, A, BIG]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=255), INVALID), (dict(_2=0), INVALID), (dict(_3=255), INVALID), (dict(_4=I8), INVALID),
    (dict(_5=3), INVALID), (dict(_5=0), INVALID), (dict(_6=0.0), INVALID), (dict(_6=-1.0), INVALID), (dict(_6=float("nan")), INVALID),
    (dict(_6=float("inf")), INVALID), (dict(_7=-1), INVALID), (dict(_8=0), INVALID), (dict(_9=0), INVALID), (dict(_10=40), INVALID),
    (dict(_11=0), INVALID), (dict(_12=68), INVALID), (dict(_13=F32), INVALID), (dict(_14=0), INVALID), (dict(_15=0), INVALID),
    (dict(_16=0), INVALID), (dict(_17=0), INVALID), (dict(_18=-1), INVALID), (dict(_18=1025), INVALID), (dict(_19=-1), INVALID),
    (dict(_20=-1), INVALID),
    # types that the tensor cores do not multiply with one another
    (dict(_4=BF16), INVALID), (dict(_13=BF16), INVALID), (dict(_4=F32, _13=BF16), INVALID),
    (dict(_0=A + 1), ALIGN), (dict(_2=A + 1), ALIGN), (dict(_8=A + 8), ALIGN), (dict(_14=A + 2), ALIGN), (dict(_16=A + 2), ALIGN),
    (dict(_17=A + 2), ALIGN), (dict(_21=A + 16), ALIGN),
    (dict(_21=0), WORKSPACE), (dict(_22=0), WORKSPACE), (dict(_22=1 << 14), WORKSPACE),
])
def test_attention(q4lib, at, code):
    refuse(q4lib, "q4_attention", change(ATTEND, **at), code)


PROBS = [A, 100, A, 100, F32, A, 4, 100]   # P, ldp, logits, ldl, type, temperature, rows, n


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=99), INVALID), (dict(_2=0), INVALID), (dict(_3=99), INVALID), (dict(_4=I8), INVALID),
    (dict(_6=-1), INVALID), (dict(_7=0), INVALID), (dict(_7=(1 << 24) + 1, _1=BIG, _3=BIG), INVALID),
    (dict(_0=A + 2), ALIGN), (dict(_2=A + 2), ALIGN), (dict(_2=A + 1, _4=F16), ALIGN), (dict(_5=A + 2), ALIGN),
])
def test_probabilities(q4lib, at, code):
    refuse(q4lib, "q4_token_probs", change(PROBS, **at), code)


# tokens, ldt, kept, P, ldp, Q, ldq, drafted, ldd, counts, accept, lda, sample, n_seq, max_draft, n
VERIFY = [A, 5, A, A, 100, A, 100, A, 4, A, A, 4, A, 2, 4, 100]


@pytest.mark.parametrize("at,code", [
    (dict(_0=0), INVALID), (dict(_1=4), INVALID), (dict(_2=0), INVALID), (dict(_3=0), INVALID), (dict(_4=99), INVALID),
    (dict(_6=99), INVALID), (dict(_7=0), INVALID), (dict(_8=3), INVALID), (dict(_10=0), INVALID), (dict(_11=3), INVALID),
    (dict(_12=0), INVALID), (dict(_13=-1), INVALID), (dict(_14=-1), INVALID), (dict(_14=1025, _1=BIG, _8=BIG, _11=BIG), INVALID),
    (dict(_15=0), INVALID), (dict(_15=(1 << 20) + 1, _4=BIG, _6=BIG), INVALID),
    (dict(_0=A + 2), ALIGN), (dict(_2=A + 2), ALIGN), (dict(_3=A + 2), ALIGN), (dict(_5=A + 2), ALIGN), (dict(_7=A + 2), ALIGN),
    (dict(_9=A + 2), ALIGN), (dict(_10=A + 2), ALIGN), (dict(_12=A + 2), ALIGN),
])
def test_verification(q4lib, at, code):
    refuse(q4lib, "q4_draft_verify", change(VERIFY, **at), code)


def test_calls_of_nothing(q4lib):
    """No sequences or no rows: nothing is asked of the addresses."""
    def call(name, good, **at):
        args = [0 if v == A else v for v in change(good, **at)]
        assert getattr(q4lib, name)(*args, stream=0, check=False) == 0

    call("q4_kv_write", WRITE, _10=0)
    call("q4_kv_write", WRITE, _16=0)
    call("q4_kv_read", READ, _15=0)
    call("q4_kv_read", READ, _16=0)
    call("q4_attention", ATTEND, _18=0)
    call("q4_attention", ATTEND, _19=0)
    call("q4_token_probs", PROBS, _6=0)
    call("q4_draft_verify", VERIFY, _13=0)
