"""Orders in the paged kernels' sources that no run can show to hold: an access that
would only sometimes come too early is looked for in the text."""
import os

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "sink_window_attention_b200", "csrc")


def test_staged_codes_are_used_before_their_place_is_written_again():
    """8-bit tile kernel: a loader reads its staged codes with plain loads and hands
    the place to an asynchronous copy, which no fence orders behind those loads. So the
    copy is issued behind the last use of what was read, and behind the buffer's
    publication, whose barrier arrival the compiler moves nothing across."""
    text = open(os.path.join(CSRC, "ll_paged_prefill.cuh")).read()
    begin = text.index("for (int kv = 0; kv < 2; ++kv)", text.index("raw0 = smem_addr(sRaw)"))
    loop = text[begin:text.index("pg = pg1;", begin)]
    assert "sRaw + (kv * STEPS + k)" in loop and loop.count("fetch(") == 1
    fetch = loop.index("fetch(kv, i + 1")
    for use in ("sRaw + (kv * STEPS + k)", "buf[k].w", "dst + off1", "publish(st)"):
        assert loop.rindex(use) < fetch, use
