// ringsim_host.h -- host helpers shared by the library's entry points: the
// RINGSIM_DEBUG log and the roctx ranges around API calls.
#pragma once

#include <dlfcn.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace ringsim {

enum LogLevel { kLogNone = 0, kLogWarn = 1, kLogInfo = 2 };

inline int log_level() {
  static const int level = [] {
    const char* e = std::getenv("RINGSIM_DEBUG");
    if (!e) return (int)kLogNone;
    if (!std::strcmp(e, "INFO")) return (int)kLogInfo;
    if (!std::strcmp(e, "WARN")) return (int)kLogWarn;
    return (int)kLogNone;
  }();
  return level;
}

#define RS_LOG(lvl, ...)                                   \
  do {                                                     \
    if (log_level() >= (lvl)) {                            \
      std::fprintf(stderr, "ringsim %s: ", (lvl) == kLogWarn ? "WARN" : "INFO"); \
      std::fprintf(stderr, __VA_ARGS__);                   \
      std::fprintf(stderr, "\n");                          \
    }                                                      \
  } while (0)

// roctx ranges around the API calls ("NCCL" book, ch. 3, s. 3.1 and the
// enqueue chapter: an NVTX mark at every API entry). With RINGSIM_ROCTX=1
// the library loads a roctx library at its first call and pushes a range
// named after the call for its duration; rocprofv3 --marker-trace shows them
// next to the kernels. Off by default, at the cost of one predictable branch
// per call; nothing is linked in.
struct Roctx {
  int (*push)(const char*) = nullptr;
  int (*pop)() = nullptr;
};

inline const Roctx& roctx() {
  static const Roctx r = [] {
    Roctx x;
    const char* e = std::getenv("RINGSIM_ROCTX");
    if (!e || !*e || !std::strcmp(e, "0")) return x;
    for (const char* lib : {"librocprofiler-sdk-roctx.so.1", "libroctx64.so.4"}) {
      void* h = dlopen(lib, RTLD_NOW | RTLD_LOCAL);
      if (!h) continue;
      x.push = reinterpret_cast<int (*)(const char*)>(dlsym(h, "roctxRangePushA"));
      x.pop = reinterpret_cast<int (*)()>(dlsym(h, "roctxRangePop"));
      if (x.push && x.pop) {
        RS_LOG(kLogInfo, "roctx ranges on (%s)", lib);
        return x;
      }
      x = Roctx{};
    }
    RS_LOG(kLogWarn, "RINGSIM_ROCTX is set but no roctx library could be loaded");
    return x;
  }();
  return r;
}

// A range for the lifetime of the object (one API call).
class RoctxRange {
 public:
  explicit RoctxRange(const char* name) : on_(roctx().push != nullptr) {
    if (on_) roctx().push(name);
  }
  ~RoctxRange() {
    if (on_) roctx().pop();
  }
  RoctxRange(const RoctxRange&) = delete;
  RoctxRange& operator=(const RoctxRange&) = delete;

 private:
  const bool on_;
};

}  // namespace ringsim
