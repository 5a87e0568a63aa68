// live_context_id against stand-ins of the driver: which calls are made, and
// what it returns, for a live context, none, one that a reset has ended, and
// an initialisation that fails or does not help.
#include <cstdio>

#include "context_id.h"

struct Driver {
  void* now;            // the thread's current context
  int dead = 0;         // handles below this address are of ended contexts
  void* after = nullptr;  // current once init has run
  int init_error = 0, inits = 0, asks = 0;
};

static int run(Driver& d, unsigned long long* id) {
  return zg::live_context_id(
      [&](void** c) { return *c = d.now, 0; },
      [&](void* c, unsigned long long* out) {
        ++d.asks;
        if ((long)c <= d.dead) return 709;
        *out = 100 + (long)c;
        return 0;
      },
      [&] {
        ++d.inits;
        if (d.init_error) return d.init_error;
        if (d.after) d.now = d.after;
        return 0;
      },
      id);
}

int main() {
  struct Case {
    const char* name;
    Driver d;
    int want, inits, asks;
    unsigned long long id;
  } cases[] = {
      {"alive", {(void*)5}, 0, 0, 1, 105},
      {"none", {nullptr, 0, (void*)6}, 0, 1, 1, 106},
      {"ended", {(void*)5, 5, (void*)7}, 0, 1, 2, 107},
      {"ended, no other", {(void*)5, 5}, -1, 1, 2, 0},
      {"none, no other", {nullptr}, -1, 1, 0, 0},
      {"init fails", {(void*)5, 5, (void*)7, 3}, 3, 1, 1, 0},
  };
  int bad = 0;
  for (Case& c : cases) {
    unsigned long long id = 0;
    const int got = run(c.d, &id);
    const bool ok = got == c.want && c.d.inits == c.inits && c.d.asks == c.asks && id == c.id;
    std::printf("%s %s\n", ok ? "ok" : "wrong", c.name);
    bad += !ok;
  }
  return bad;
}
