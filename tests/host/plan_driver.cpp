// Host-only driver around the planners of the attention half's kernels (PLANNER: the source
// that holds one): reads sizes from standard input, a call a line, and prints the plan
// that a device of 256 CUs gets for each.  No kernel and no HIP call runs.
#include PLANNER

#include <cstdio>

extern "C" {  // what the sources' kernels would register
const char __hip_fatbin[8] = {};
void** __hipRegisterFatBinary(const void*) {
  static void* module;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
}

int main() {
  twl::DeviceInfo dev;
  dev.cu_count = 256;
  long v[8];
#ifdef ATTENTION  // T B group n_kv D table_keys window sinks -> small large small_rows splits large_splits
  while (std::scanf("%ld%ld%ld%ld%ld%ld%ld%ld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7) == 8) {
    const twl::Plan p = twl::make_plan(v[0], v[1], static_cast<int>(v[2]), static_cast<int>(v[3]), static_cast<int>(v[4]), v[5],
                                       static_cast<int>(v[6]), static_cast<int>(v[7]), dev);
    std::printf("%d %d %d %d %d\n", p.small, p.large, p.small_rows, p.splits, p.large_splits);
  }
#else  // M N K -> rt mt tile splits
  while (std::scanf("%ld%ld%ld", v, v + 1, v + 2) == 3) {
    const twl::Plan p = twl::make_plan(v[0], v[1], v[2], dev);
    std::printf("%d %d %d %d\n", p.rt, p.mt, p.tile, p.splits);
  }
#endif
}
