// Who has been told of the block operators' expired waits.  The kernels' status word is one for a device and is cleared
// by the first thread that reads it; the count behind it lets every other thread learn of the same wait.
#pragma once
#include <atomic>

namespace mrf {

struct ExpiredWaits {
  std::atomic<unsigned> count{0}, site{0};
  // The device's word was set (and has been cleared).
  void found(unsigned at) {
    site.store(at);
    count.fetch_add(1);
  }
  // Whether one was found since this thread last asked; `seen` is the thread's own, 0 before it first asks.
  bool since(unsigned &seen) {
    const unsigned now = count.load();
    const bool some = now != seen;
    seen = now;
    return some;
  }
};

}  // namespace mrf
