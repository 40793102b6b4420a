// workspace_turn.h -- calls that share a workspace enqueue their launches one after the other.
#pragma once

#include <condition_variable>
#include <mutex>

namespace muon {

// Held while the launches of one call are enqueued that leave something in its workspace: a later
// launch of the call reads it, and calls of every kind share the workspace that the binding keeps
// for a stream, so that no other thread's launches may come between.  Calls on other workspaces do
// not wait, whatever a launch of this one waits for (a full queue, behind it another device).  A
// call that leaves nothing gives null and holds nothing.
class WorkspaceTurn {
 public:
  explicit WorkspaceTurn(const void* workspace) : workspace_(workspace) {
    if (!workspace_) return;
    std::unique_lock<std::mutex> lk(mu_);
    if (taken()) {
      ++waiting_;
      cv_.wait(lk, [this] { return !taken(); });
      --waiting_;
    }
    next_ = holders_;
    holders_ = this;
  }
  ~WorkspaceTurn() {
    if (!workspace_) return;
    bool wake;
    {
      std::lock_guard<std::mutex> lk(mu_);
      WorkspaceTurn** p = &holders_;
      while (*p != this) p = &(*p)->next_;
      *p = next_;
      wake = waiting_ > 0;
    }
    if (wake) cv_.notify_all();
  }
  WorkspaceTurn(const WorkspaceTurn&) = delete;
  WorkspaceTurn& operator=(const WorkspaceTurn&) = delete;

 private:
  bool taken() const {                       // (a list as long as there are threads in calls)
    for (const WorkspaceTurn* t = holders_; t; t = t->next_)
      if (t->workspace_ == workspace_) return true;
    return false;
  }
  const void* const workspace_;
  WorkspaceTurn* next_ = nullptr;
  static inline std::mutex mu_;              // of the list, never held over a launch
  static inline std::condition_variable cv_;
  static inline WorkspaceTurn* holders_ = nullptr;
  static inline int waiting_ = 0;
};

}  // namespace muon
