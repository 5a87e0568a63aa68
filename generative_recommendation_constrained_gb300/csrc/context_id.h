// The unique id of the calling thread's current CUDA context, by whatever
// calls it is given (engine.cpp: the driver's; the tests: stand-ins).
#pragma once

namespace zg {

// current(void** ctx) and id_of(void* ctx, id*) return 0 for success, init()
// makes the device's primary context current (0 for success).  A context that
// is current and alive is asked at once: init takes longer than a launch.
// Where there is none, or the handle is of one that a reset has ended, init
// comes first and both are asked once more.  Returns 0, init's error, or -1.
template <typename Current, typename IdOf, typename Init>
int live_context_id(Current current, IdOf id_of, Init init, unsigned long long* id) {
  auto ask = [&]() {
    void* ctx = nullptr;
    return current(&ctx) == 0 && ctx && id_of(ctx, id) == 0;
  };
  if (ask()) return 0;
  if (const int e = init()) return e;
  return ask() ? 0 : -1;
}

}  // namespace zg
