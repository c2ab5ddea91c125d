// device_scope.h -- make a device the calling thread's current one for a scope, and
// give the thread its own back at the end. Runtime: get(int *) and set(int), 0 for
// success (a test gives plain functions).
#pragma once

template <class Runtime>
class DeviceScope {
    int was = -1;  // the device to go back to, -1: nothing to do (declared first: enter() sets it)

    int enter(int device)
    {
        int cur = -1;
        int e = Runtime::get(&cur);
        if (e == 0 && cur != device && (e = Runtime::set(device)) == 0)
            was = cur;
        return e;
    }

public:
    const int err;  // not 0: the device could not be made current

    explicit DeviceScope(int device) : err(enter(device)) {}
    ~DeviceScope()
    {
        if (was >= 0)
            Runtime::set(was);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
};
