#!/bin/bash
# Builds tests/native/_build/abi_exercise and rows_exercise (the row operators):
# the library sources and the ABI exercise drivers with AddressSanitizer and UndefinedBehaviorSanitizer on the
# host code only (each -fsanitize= sits behind -Xarch_host; the gfx950 device
# code is compiled as in the library build, without sanitizers).  The objects
# are linked statically into each executable, so the sanitizer runtime is part
# of the program.  Run them on a machine with an MI355X (rows_exercise also runs
# without one, and then stops before the calls that launch):
#   ASAN_OPTIONS=detect_leaks=0:halt_on_error=1:verify_asan_link_order=0 \
#   UBSAN_OPTIONS=halt_on_error=1:print_stacktrace=1 tests/native/_build/abi_exercise
#   (and the same for rows_exercise)
# detect_leaks=0: the HIP runtime keeps allocations until exit by design.
set -euo pipefail
HERE="$(cd "$(dirname "${BASH_SOURCE[0]}")" && pwd)"
ROOT="$(cd "$HERE/../.." && pwd)"
CSRC="$ROOT/soft_clustering_amd/csrc"
OUT="$HERE/_build"
mkdir -p "$OUT"
HIPCC=/opt/rocm/bin/hipcc
CLANG=/opt/rocm/llvm/bin/clang++
# -O3 and the target features of the library build, so the device code is the same
COMMON=(--offload-arch=gfx950 -O3 -std=c++17 -I "$ROOT/include"
        -Xclang -target-feature -Xclang -packed-fp32-ops)
SAN=(-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined
     -Xarch_host -fno-sanitize-recover=undefined -Xarch_host -fno-omit-frame-pointer -Xarch_host -g)
# an object is rebuilt when it is missing or older than its source or a header
stale() {
  local o="$1" s="$2" h
  [ -s "$o" ] || return 0
  for h in "$s" "$CSRC"/*.h "$ROOT"/include/*.h; do [ "$h" -nt "$o" ] && return 0; done
  return 1
}
objs=()
for src in gmm_kernels gmm_assign gmm_lists gmm_api gmm_mx gmm_byte gmm_draw gmm_losses gmm_rows_api; do
  if stale "$OUT/$src.o" "$CSRC/$src.hip"; then
    rm -f "$OUT/$src.o"
    "$HIPCC" "${COMMON[@]}" "${SAN[@]}" -c "$CSRC/$src.hip" -o "$OUT/$src.o" 2> "$OUT/$src.log" &
  fi
  objs+=("$OUT/$src.o")
done
for exe in abi_exercise rows_exercise; do
  if stale "$OUT/$exe.o" "$HERE/$exe.cpp"; then
    rm -f "${OUT:?}/${exe:?}.o"
    "$HIPCC" "${COMMON[@]}" "${SAN[@]}" -x hip -c "$HERE/$exe.cpp" -o "$OUT/$exe.o" 2> "$OUT/$exe.log" &
  fi
done
wait
for o in "${objs[@]}" "$OUT/abi_exercise.o" "$OUT/rows_exercise.o"; do
  [ -s "$o" ] || { echo "compile failed: $o" >&2; grep -i error "${o%.o}.log" >&2; exit 1; }
done
# host link: objects only, the sanitizer runtimes linked statically
for exe in abi_exercise rows_exercise; do
  "$CLANG" -fsanitize=address,undefined -o "$OUT/$exe" "$OUT/$exe.o" "${objs[@]}" \
    -L/opt/rocm/lib -Wl,-rpath,/opt/rocm/lib -lamdhip64
  echo "built $OUT/$exe"
done
