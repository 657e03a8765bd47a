"""Where the wide prefix-attention kernel keeps things in shared memory, read
from its source: what one warp may still read while another one writes must
not lie in the same bytes."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_diffusion_speculative_hidden_gb300", "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _layout(dh):
    """The integer constants of WideLayout<dh>."""
    names = {"DH": dh, "true": 1, "false": 0}
    for src in (_code("prefix_common.cuh"), _code("prefix_wide.cu")):
        names.update((n, int(v)) for n, v in re.findall(r"constexpr int (kWide\w+) = (\d+);", src))
    names.update(kPage=16)
    names["kWidePages"] = names["kWideKeys"] // 16
    body = re.search(r"struct WideLayout \{(.*?)\n\};", _code("prefix_wide.cu"), re.S).group(1)
    for decl in re.findall(r"static constexpr \w+ ([^;]*);", body):
        for name, value in re.findall(r"(\w+) = ((?:[^,()]|\([^()]*\))*)", decl):
            value = re.sub(r"(.+?)==(.+?)\?(.+?):(.+)", r"(\3) if \1==\2 else (\4)", value)
            value = re.sub(r"^(\w+) \?(.+?):(.+)", r"(\2) if \1 else (\3)", value)
            names[name] = eval(value.replace("/", "//"), {}, names)
    return names


@pytest.mark.parametrize("dh", [64, 128])
def test_tokens_of_a_packed_tile_share_no_bytes_with_what_the_softmax_writes(dh):
    """The softmax warps of a packed tile read its token list after the last barrier of the CTA; the
    row maxima and sums that the first of them exchange in pairs must not be written over it."""
    L = _layout(dh)
    kernel = _code("prefix_wide.cu")

    def place(name):
        at = re.search(r"\* ?%s = reinterpret_cast<\w+\*>\((.*?)\);" % name, kernel).group(1)
        if at == "red":
            return place("red")
        return L[re.fullmatch(r"smem \+ L::(\w+)", at).group(1)]
    red, red_bytes = place("red"), 2 * L["SOFT"] * 32 * 4
    tokens, token_bytes = place("tokens"), L["kWideTile"] * 4
    assert tokens + token_bytes <= red or red + red_bytes <= tokens
    assert tokens >= L["OFF_BAR"] + 256 and tokens + token_bytes <= L["SMEM"] - 1024
