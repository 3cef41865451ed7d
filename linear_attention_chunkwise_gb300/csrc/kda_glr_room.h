// kda_glr_room.h -- what the launches of the gated linear recurrence keep about a device: how many clusters of a kernel fit it.
#pragma once

#include <atomic>

namespace kda {

constexpr int kGlrMaxCluster = 16;  // blocks of a cluster

// How many clusters of 1, 2 .. blocks of a kernel find room beside each other.
struct GlrRoom {
    int clusters[kGlrMaxCluster + 1] = {};
};

// A kernel's rooms by device.  Host threads that come before a device's is known each look for themselves, into a table of their own; the
// first one done leaves it for later calls, and it is never written again, so a call's clusters do not depend on who else is calling.
class GlrRooms {
   public:
    // look(&room) fills a table of `dev` and gives 0, or an error, which is not kept.
    template <typename F>
    auto get(int dev, const F& look, GlrRoom* out) -> decltype(look(out)) {
        Slot* slot = dev >= 0 && dev < kDevices ? &slots_[dev] : nullptr;  // devices beyond look every time
        if (slot && slot->state.load(std::memory_order_acquire) == kKnown) {
            *out = slot->room;
            return {};
        }
        const auto err = look(out);
        int state = kNone;
        if (!err && slot && slot->state.compare_exchange_strong(state, kWritten, std::memory_order_relaxed)) {
            slot->room = *out;
            slot->state.store(kKnown, std::memory_order_release);
        }
        return err;
    }

   private:
    static constexpr int kDevices = 64, kNone = 0, kWritten = 1, kKnown = 2;
    struct Slot {
        std::atomic<int> state{kNone};
        GlrRoom room;
    };
    Slot slots_[kDevices];
};

}  // namespace kda
