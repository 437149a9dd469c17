"""Calls of the BF16 paged cache's attention for each way their work is shared out, found
by the library's own rules for the GPU at hand, so that a later change of the rules
cannot lead the tests elsewhere."""
from . import cache_plain as plain


def form_of(lynx, counts, kv, H_q, H_kv, page, decode, pages, sms):
    table, _ = plain.table_for(kv, page, 0, 0, pages)
    return lynx.lynx_cache_attn_form(sum(counts), len(counts), counts[0] if decode else 0, H_q,
                                     H_kv, 128, page, table.shape[1], sms)


def parts_case(lynx, sms, counts, kv, G, page, pages, absent=False):
    """(counts, kv, H_q, H_kv, page, False, pages) with the smallest H_kv for which
    the last units are cut in parts; `absent`: so many that some of them are units of
    the bound on their number, not of the call."""
    blocks = sum(-(-n * G // 256) for n in counts)
    for H_kv in range(1, 200):
        case = (counts, kv, G * H_kv, H_kv, page, False, pages)
        if form_of(lynx, *case, sms) != lynx.LYNX_CACHE_PARTS:
            continue
        units = (sum(counts) * G // 256 + len(counts)) * H_kv
        last = units % min(sms, 160)
        there = last - (units - blocks * H_kv)           # of the last units, those of the call
        if there >= (1 if absent else last) and (not absent or there < last):
            return case
    raise AssertionError("no such case: the rules have changed")


def parts_cases(lynx, sms):
    return {
        # two parts' worth of long contexts
        "long": parts_case(lynx, sms, [300, 301], [2600, 2500], 1, 64, None),
        # fewer tiles than parts: parts without a tile
        "short last": parts_case(lynx, sms, [300, 301], [2600, 301], 1, 256, None),
        # rows that see nothing in the last units
        "negative": parts_case(lynx, sms, [300, 301], [2600, 40], 1, 64, None),
        "nothing": parts_case(lynx, sms, [300, 301], [2600, 0], 1, 128, None),
        # blocks of the grid behind the last unit
        "absent": parts_case(lynx, sms, [300, 0, 301], [2300, 9, 700], 2, 512, None, absent=True),
        # a second half with few rows, several query heads to a row block
        "heads": parts_case(lynx, sms, [130, 161], [900, 2200], 4, 64, 40),
    }


# several units to a CTA, of one and of both row halves, of one and of several tiles,
# sequences without tokens and without keys among them
TAKEOVER = ([300, 0, 513, 65, 700, 1, 130, 4], [300, 5, 1900, 65, 701, 1, 1000, 0], 80, 40, 64,
            False, 32)
