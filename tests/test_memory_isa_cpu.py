"""Which instructions the kernels reach memory with (host only: hipcc cross-compiles).

Allow-lists over the gfx950 assembly of every kernel source: data leaves a wave through
vector stores and LDS alone, scalar instructions read memory and never write it, and
the atomics are the integer ones in LDS.
"""
import importlib.util
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location(
    "_zs_build_memory", os.path.join(ROOT, "zero_sharded_mixed_shard_amd", "build.py"))
build = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(build)

# scalar instructions: those between registers, of control, and the loads
SCALAR = re.compile(
    r"s_(add|addc|addk|and|andn1|andn2|ashr|barrier|bcnt0|bcnt1|bfe|bfm|bitcmp0|bitcmp1|bitset0|"
    r"bitset1|branch|brev|cbranch|cmov|cmp|cmpk|cselect|endpgm|ff0|ff1|flbit|getpc|lshl|lshl1|"
    r"lshl2|lshl3|lshl4|lshr|max|min|mov|movk|mul|mulk|nand|nop|nor|not|or|orn1|orn2|pack|"
    r"setpc|setprio|sext|sleep|sub|subb|swappc|wqm|waitcnt|xnor|xor)(_\w+)?|s_load_dword(x2|x4|x8|x16)?")
VECTOR = re.compile(r"(global|scratch)_(load|store)_(u?byte|sbyte|u?short|sshort|dword|dwordx[234])"
                    r"(_d16)?(_d16_hi)?")
LDS = re.compile(r"ds_(read|write)\w*|ds_(add|or|max|min)_[ui]32|ds_(b?permute|swizzle)_b32")


@pytest.mark.parametrize("src", build.KERNEL_SOURCES)
def test_memory_is_reached_by_known_instructions(src):
    names = set(re.findall(r"^\s+((?:s|ds|global|scratch|flat|buffer|tbuffer|image)_\w+)\s",
                           build.device_assembly(src), re.M))
    assert {"global_store_dwordx4", "s_waitcnt"} <= names
    unknown = [n for n in names
               if not (SCALAR.fullmatch(n) or VECTOR.fullmatch(n) or LDS.fullmatch(n))]
    assert not unknown, sorted(unknown)
