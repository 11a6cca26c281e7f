"""Launches of the attention with rules that are too large: refused on the
host, whichever of a call's launches it is."""
from bigvgan_waveform_decoder_amd import avae
from tests.test_rope_host import ESHAPE, _attn, _cache, _rows


def test_joins_are_counted_by_sequence():
    """With rules a join has a row of workgroups for each sequence, as many as
    the most rows that one may have: 1024 sequences of up to 16 rows, 4096
    heads, four rows a workgroup are 2^24, though there are 16 rows in all."""
    cache = _cache(n=4096, heads=4096)
    rows = _rows(cols=16, ld=16, seqs=1024, total=16, max_rows=16)
    assert _attn(cache=cache, rows=rows, heads=4096, tok=4096 * 64, max_len=256) == ESHAPE
    assert b"1024 sequences of up to 16 rows are 16777" in avae.lib().avae_last_error()
