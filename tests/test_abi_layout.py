"""The structures, types and argument lists by which ctypes calls the objectives
are the C header's: compared with a C program's offsets and the header's own
declarations. CPU only."""
import ctypes
import os
import re
import subprocess

import pytest

import row_wise_softmax_ce_gb300 as ce
from row_wise_softmax_ce_gb300 import build as cuda_build

STRUCTS = {"ce_policy": ce.Policy, "ce_preference": ce.Preference}


@pytest.fixture(scope="module")
def header():
    with open(ce.HEADER) as f:
        return re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)


def test_structures(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        for field, _ in cls._fields_:
            lines.append(f'printf("{name}.{field} %zu %zu\\n", offsetof({name}, {field}), sizeof((({name} *)0)->{field}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ce_rows.h"\nint main(void)\n{\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(ce.HEADER), str(src), "-o", exe], check=True)
    want = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    got = []
    for name, cls in STRUCTS.items():
        got.append(f"{name} {ctypes.sizeof(cls)}")
        got += [f"{name}.{f} {getattr(cls, f).offset} {getattr(cls, f).size}" for f, _ in cls._fields_]
    assert got == want


@pytest.mark.parametrize("name", STRUCTS)
def test_every_field(header, name):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), header, re.S).group(1)
    fields = []
    for kind, names in re.findall(r"(double|int)\s+([^;]+);", body):
        fields += [(n.strip(), ctypes.c_double if kind == "double" else ctypes.c_int) for n in names.split(",")]
    assert fields == STRUCTS[name]._fields_


def test_preference_kinds(header):
    body = re.search(r"enum ce_preference_kind \{(.*?)\}", header, re.S).group(1)
    kinds = dict(re.findall(r"CE_PREF_(\w+) = (\d+)", body))
    assert {k.lower(): int(v) for k, v in kinds.items()} == ce.PREFERENCE_KINDS


@pytest.mark.parametrize("name", ["logp_rows", "policy_loss", "policy_step", "preference_loss", "preference_step"])
def test_arguments(header, name):
    cuda_build.build()
    args = re.search(r"CE_API int %s\((.*?)\);" % name, header, re.S).group(1).split(",")

    def kind(arg):
        if "*" in arg or "ce_stream_t" in arg:
            return ctypes.c_void_p
        return {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "double": ctypes.c_double}[arg.split()[0]]
    assert [kind(a) for a in args] == list(getattr(ce.lib(), name).argtypes)
